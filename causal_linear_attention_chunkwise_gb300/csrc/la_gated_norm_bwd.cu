// la_gated_norm_bwd.cu -- backward pass of the norm and gate of a layer's heads.
//
// With a = act(gate), a' its derivative, and (mean, r, n) the row's norm:
//
//     y = (n w + b) a:       g = dy a w,  dgate = dy (n w + b) a',  dw = sum dy a n,
//                            db = sum dy a,  dx = r (g - mean(g) - n mean(g n))
//     y = norm(x a) w + b:   g = dy w,  u = r (g - mean(g) - n mean(g n)),  dx = u a,
//                            dgate = u x a',  dw = sum dy n,  db = sum dy
//
// Nothing of the forward pass is kept: x and the gate give everything again.
//
// Wide rows are bound by the bytes (2 x 2047 x 4096 fp32: 57 us, 5.9 TB/s); 64-value rows by
// instructions, an exponential and a reciprocal an element among them (4 x 16 x 4096 x 64 bf16:
// 38 us, 4.4 TB/s).
#include <cstdint>

#include "la_block_norm_bwd.cuh"

namespace la {
namespace {

// sigmoid(z) and 1 - sigmoid(z) of a cell of values.  With e = e^-z they are 1 / (1 + e) and
// e / (1 + e); as a difference from 1 the second would lose its digits above z = 10.  Where e
// overflows the sigmoid is 0 and what its complement is multiplied by as well.
constexpr float kMostExp = 0x1p126f;
__device__ __forceinline__ void sigmoid_both(float z, float &s, float &rest) {
  const float e = ex2_approx(-z * kLog2e);
  s = rcp_approx(1.f + e);
  rest = fminf(e, kMostExp) * s;
}
__device__ __forceinline__ void sigmoid_both(unsigned long long z, unsigned long long &s,
                                             unsigned long long &rest) {
  float a, b, x, y;
  unpack2(mul2(z, dup2(-kLog2e)), a, b);
  a = ex2_approx(a), b = ex2_approx(b);
  unpack2(add2(pack2(a, b), dup2(1.f)), x, y);
  s = pack2(rcp_approx(x), rcp_approx(y));
  rest = mul2(pack2(fminf(a, kMostExp), fminf(b, kMostExp)), s);
}

// act(z) and its derivative, with s = sigmoid(z): z s has s + z s (1 - s).
template <int ACT, int V, typename C>
__device__ __forceinline__ void act_and_slope(C z, C &a, C &slope) {
  if constexpr (ACT == LA_ACT_NONE) {
    a = z, slope = CellOf<V>::both(1.f);
  } else {
    C s, rest;
    sigmoid_both(z, s, rest);
    a = ACT == LA_ACT_SILU ? mul2(z, s) : s;
    slope = ACT == LA_ACT_SILU ? fma2(a, rest, s) : mul2(s, rest);
  }
}

// Weights shared by the heads: the rows are those of all heads, in the order of
// the tokens.  Weights of each head: a block stays with head blockIdx.y.
// BIAS: there is a bias, or a gradient of one.  FIRST: there is a gate, in front of the norm.
// Blocks of teams to an SM: three where their registers allow it (4 x 16 x 4096 x 64 bf16: 38 us, with
// two 40).
template <int V, int LANES, int I, bool BIAS, bool FIRST> constexpr int kBlocksPerSm =
    LANES ? (I == 1 && (V <= 4 || !(BIAS || FIRST)) ? 3 : 2) : 1;

template <typename T, int V, int LANES, int I, bool BIAS, bool FIRST, int MAXT>
__global__ void __launch_bounds__(MAXT, kBlocksPerSm<V, LANES, I, BIAS, FIRST>)
gated_norm_bwd_kernel(const GatedNormBwdArgs a, long long rows, float *part) {
  using P = Cells<V>;
  using C = typename P::C;
  constexpr int H = P::H, N = H * I;
  __shared__ float red[2][4][32];
  __shared__ float sum[LANES ? kNormTeamThreads / 32 * LANES * V * I : 1];
  const int size = LANES ? LANES : blockDim.x;
  const int lane = LANES ? threadIdx.x % LANES : threadIdx.x;
  const int teams = LANES ? kNormTeamThreads / size : 1;
  const long long step = (long long)gridDim.x * teams;
  long long r = (long long)blockIdx.x * teams + (LANES ? threadIdx.x / size : 0);
  const int d = a.d, own_head = a.weight_heads > 1 ? (int)blockIdx.y : -1;
  const float inv = 1.f / d;
  const bool gate = FIRST || a.gate;
  const bool layer = a.norm == LA_NORM_LAYER;
  auto both = [](float v) { return CellOf<V>::both(v); };
  auto total = [](C c) { return CellOf<V>::sum(c); };
  int turn = 0;
  Raw<T, V> x[I], z[I], dy[I];
  // Row r's head and token, carried along: a step adds (db, dt, dh), without divisions.  t is
  // unsigned: a step past a sequence's end may take it to 2^31 and above.
  struct Place {
    long long b, bt;
    unsigned t;
    int h;
  };
  auto split = [&](long long row) {
    Place p;
    p.bt = own_head >= 0 ? row : div_index(row, a.H);
    p.h = own_head >= 0 ? own_head : (int)(row - p.bt * a.H);
    p.b = div_index(p.bt, a.L);
    p.t = (unsigned)(p.bt - p.b * a.L);
    return p;
  };
  const Place stride = [&] {
    Place p = split(step);
    if (own_head >= 0) p.h = 0;
    return p;
  }();
  auto advance = [&](Place p) {
    p.h += stride.h, p.bt += stride.bt, p.t += stride.t, p.b += stride.b;
    if (own_head < 0 && p.h >= a.H) p.h -= a.H, ++p.bt, ++p.t;
    if (p.t >= (unsigned)a.L) p.t -= a.L, ++p.b;
    return p;
  };
  auto fetch = [&](const Place &p) {
    const T *xr = static_cast<const T *>(a.x) + p.b * a.x_bs + p.h * a.x_hs + p.t * a.x_ts;
    const T *zr = static_cast<const T *>(a.gate) + p.bt * a.gate_stride + (long long)p.h * d;
    const T *yr = static_cast<const T *>(a.dy) + p.bt * a.dy_stride + (long long)p.h * d;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = (lane + i * size) * V;
      if (c >= d) continue;
      x[i] = load_raw<T, V>(xr + c);
      if (gate) z[i] = load_raw<T, V>(zr + c);
      dy[i] = load_raw<T, V>(yr + c);
    }
  };
#pragma unroll
  for (int i = 0; i < I; ++i) x[i] = z[i] = dy[i] = Raw<T, V>{};
  C w[N], bias[BIAS ? N : 1], dw[N], db[BIAS ? N : 1];
  const long long w0 = own_head >= 0 ? (long long)own_head * d : 0;
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int c = (lane + i * size) * V;
    float f[V];
    params_or<V>(a.weight ? a.weight + w0 : nullptr, c, d, 1.f, f);
    P::pack(f, w + i * H);
    if constexpr (BIAS) {
      params_or<V>(a.bias ? a.bias + w0 : nullptr, c, d, 0.f, f);
      P::pack(f, bias + i * H);
    }
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    dw[j] = C(0);
    if constexpr (BIAS) db[j] = C(0);
  }
  Place at = split(r < rows ? r : 0);
  if (r < rows) fetch(at);
  // A team out of rows stays while another of its warp has one: the sums need
  // the whole warp.
  for (long long first = r - (LANES ? threadIdx.x % 32 / size : 0); first < rows;
       first += step, r += step) {
    const bool live = r < rows;
    T *dxr = static_cast<T *>(a.dx) + at.b * a.dx_bs + at.h * a.dx_hs + at.t * a.dx_ts;
    T *dzr = static_cast<T *>(a.dgate) + at.bt * a.dgate_stride + (long long)at.h * d;
    C v[N], act[N], g[N];
    C keep[N];  // what dgate has beside n: act's slope, times x where the gate comes first, else dy
#pragma unroll
    for (int i = 0; i < I; ++i) {
      float f[V];
      x[i].unpack(f);
      P::pack(f, v + i * H);
      dy[i].unpack(f);
      P::pack(f, g + i * H);
      z[i].unpack(f);
      P::pack(f, act + i * H);
    }
    auto activate_all = [&](auto kind) {
#pragma unroll
      for (int j = 0; j < N; ++j)
        act_and_slope<decltype(kind)::value, V>(act[j], act[j], keep[j]);
    };
    if (!gate) {
#pragma unroll
      for (int j = 0; j < N; ++j) act[j] = both(1.f), keep[j] = C(0);
    } else if (a.act == LA_ACT_SILU) {
      activate_all(IntC<LA_ACT_SILU>{});
    } else if (a.act == LA_ACT_SIGMOID) {
      activate_all(IntC<LA_ACT_SIGMOID>{});
    } else {
      activate_all(IntC<LA_ACT_NONE>{});
    }
    if (r + step < rows) {
      at = advance(at);
      fetch(at);
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      keep[j] = mul2(keep[j], FIRST ? v[j] : g[j]);
      if (FIRST) v[j] = mul2(v[j], act[j]);
      else g[j] = mul2(g[j], act[j]);  // the gradient of n w + b
    }
    if (layer) {
      C m0 = C(0);
#pragma unroll
      for (int j = 0; j < N; ++j) m0 = add2(m0, v[j]);
      float m[1] = {total(m0)};
      team_sums<LANES>(m, red, turn);
      const C off = both(-m[0] * inv);
#pragma unroll
      for (int i = 0; i < I; ++i)
#pragma unroll
        for (int k = 0; k < H; ++k)
          v[i * H + k] = (lane + i * size) * V < d ? add2(v[i * H + k], off) : C(0);
    }
    C q0 = C(0), q1 = C(0), q2 = C(0);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const C gw = mul2(g[j], w[j]);
      q0 = fma2(v[j], v[j], q0);
      q1 = fma2(gw, v[j], q1);
      if (layer) q2 = add2(q2, gw);
    }
    float s[2] = {total(q0), total(q1)}, mean = 0.f;
    if (layer) {
      float s3[3] = {s[0], s[1], total(q2)};
      team_sums<LANES>(s3, red, turn);
      s[0] = s3[0], s[1] = s3[1], mean = s3[2] * inv;
    } else {
      team_sums<LANES>(s, red, turn);
    }
    const float rs = rsqrtf(fmaf(s[0], inv, a.eps));
    const C rho = both(rs), against = both(-s[1] * inv * rs * rs), mean_g = both(-mean);
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = (lane + i * size) * V;
      C ox[H], oz[H];
#pragma unroll
      for (int k = 0; k < H; ++k) {
        const int j = i * H + k;
        const C n = mul2(v[j], rho);
        C u = fma2(g[j], w[j], mul2(against, v[j]));
        if (layer) u = add2(u, mean_g);
        u = mul2(rho, u);
        if (live) {
          dw[j] = fma2(g[j], n, dw[j]);
          if constexpr (BIAS) db[j] = add2(db[j], g[j]);
        }
        ox[k] = FIRST ? mul2(u, act[j]) : u;
        C y;
        if constexpr (BIAS) y = fma2(n, w[j], bias[j]);
        else y = mul2(n, w[j]);
        oz[k] = mul2(FIRST ? u : y, keep[j]);
      }
      if (!live || c >= d) continue;
      float f[V];
      P::unpack(ox, f);
      store_vec<T, V>(dxr + c, f);
      if (gate) {
        P::unpack(oz, f);
        store_vec<T, V>(dzr + c, f);
      }
    }
  }
  if (!part) return;
  const long long width = (long long)a.weight_heads * d;
  float *mine = part + (long long)blockIdx.x * width + w0;
  float f[V * I];
  if (a.dweight) {
#pragma unroll
    for (int i = 0; i < I; ++i) P::unpack(dw + i * H, f + i * V);
    block_share<V, LANES, I>(f, mine, d, sum);
    mine += (long long)gridDim.x * width;
  }
  if constexpr (BIAS) {
    if (a.dbias) {
#pragma unroll
      for (int i = 0; i < I; ++i) P::unpack(db + i * H, f + i * V);
      block_share<V, LANES, I>(f, mine, d, sum);
    }
  }
}

template <typename T, int V>
cudaError_t launch_v(const GatedNormBwdArgs &a) {
  const bool per_head = a.weight_heads > 1;
  const long long rows = (long long)a.B * a.L * (per_head ? 1 : a.H);
  const int sums = (a.dweight != nullptr) + (a.dbias != nullptr);
  const int width = a.weight_heads * a.d;
  return with_bwd_team<V>(a.d, [&](auto lanes, auto items, auto most, int threads) {
    constexpr int LANES = decltype(lanes)::value, I = decltype(items)::value;
    constexpr int MAXT = decltype(most)::value;
    const int heads = per_head ? a.H : 1, teams = LANES ? kNormTeamThreads / LANES : 1;
    const int block = LANES ? kNormTeamThreads : threads;
    float *part = sums ? static_cast<float *>(a.workspace) : nullptr;
    unsigned blocks = 0;
    auto launch = [&](auto bias, auto first) {
      constexpr bool BIAS = decltype(bias)::value != 0, FIRST = decltype(first)::value != 0;
      blocks = norm_bwd_blocks((rows + teams - 1) / teams,
                               LANES ? kBlocksPerSm<V, LANES, I, BIAS, FIRST> : 512 / block, heads);
      gated_norm_bwd_kernel<T, V, LANES, I, BIAS, FIRST, MAXT>
          <<<dim3(blocks, heads), block, 0, a.stream>>>(a, rows, part);
    };
    const bool first = a.gate && a.gate_first;
    if (a.bias || a.dbias) first ? launch(IntC<1>{}, IntC<1>{}) : launch(IntC<1>{}, IntC<0>{});
    else first ? launch(IntC<0>{}, IntC<1>{}) : launch(IntC<0>{}, IntC<0>{});
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !sums) return e;
    WeightSums w{part, (int)blocks, width, {}};
    int n = 0;
    if (a.dweight) w.out[n++] = a.dweight;
    if (a.dbias) w.out[n++] = a.dbias;
    return launch_weight_sums(w, n, a.stream);
  });
}

template <typename T>
cudaError_t launch_t(const GatedNormBwdArgs &a) {
  constexpr int V = Pack16<T>::N;
  auto fits = [](const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  auto heads_fit = [&](long long b, long long h, long long t) {
    return (a.B == 1 || b % V == 0) && (a.H == 1 || h % V == 0) && (a.L == 1 || t % V == 0);
  };
  const bool wide = a.d % V == 0 && fits(a.x) && fits(a.dx) && fits(a.gate) && fits(a.dgate) &&
                    fits(a.dy) && heads_fit(a.x_bs, a.x_hs, a.x_ts) &&
                    heads_fit(a.dx_bs, a.dx_hs, a.dx_ts) && a.dy_stride % V == 0 &&
                    (!a.gate || (a.gate_stride % V == 0 && a.dgate_stride % V == 0));
  return wide ? launch_v<T, V>(a) : launch_v<T, 1>(a);
}

}  // namespace

size_t gated_norm_bwd_workspace_bytes(int B, int H, int L, int d, int weight_heads) {
  const long long rows = (long long)B * L * (weight_heads > 1 ? 1 : H);
  const int heads = weight_heads > 1 ? H : 1;
  return 2 * sizeof(float) * norm_bwd_blocks(rows, kNormMostBlocks, heads) * (size_t)weight_heads * d;
}

cudaError_t launch_gated_norm_bwd(const GatedNormBwdArgs &a) {
  return a.dtype == LA_F32 ? launch_t<float>(a) : launch_t<__nv_bfloat16>(a);
}

}  // namespace la
