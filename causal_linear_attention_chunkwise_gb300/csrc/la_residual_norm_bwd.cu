// la_residual_norm_bwd.cu -- backward pass of the residual step between two blocks.
//
//     u = norm(x) p,  r = residual + alpha s u,  y = norm(r) w + b
//
// gives, from the gradients dy of y and dr of r (the residual stream's, from the
// blocks behind), with (rho, n) and (rho_x, n_x) the two norms,
//
//     dresidual = rho (dy w - mean(dy w) - n mean(dy w n)) + dr =: e
//     dw = sum dy n,  db = sum dy,  ds = sum alpha e u,  dp = sum alpha s e n_x
//     dx = rho_x (g - mean(g) - n_x mean(g n_x)),  g = alpha s p e   (no p: g)
//
// in one pass over dy, r, dr and x.  The means of x, r and g belong to layer norm
// alone.  r is read as the forward pass stored it.  ds and dp are alpha p and alpha s times
// one sum over rows, of e n_x (x itself without a post norm).
//
// The bytes bound it: 16384 x 4096, fp32 residual, post norm and scale, takes 201 us, 6.0 TB/s
// (sums of their own for ds and dp, when it took 236: 278).
#include <cstdint>

#include "la_block_norm_bwd.cuh"

namespace la {
namespace {

// X: x is read (a post norm, or a scale's gradient).
template <typename T, typename R, int V, int LANES, int I, bool X, int MAXT>
__global__ void __launch_bounds__(MAXT, LANES ? 2 : 1)
residual_norm_bwd_kernel(const ResidualNormBwdArgs a, float *part) {
  constexpr int RV = V < Pack16<R>::N ? V : Pack16<R>::N, RN = V / RV;
  using P = Cells<V>;
  using C = typename P::C;
  constexpr int H = P::H, N = H * I;
  __shared__ float red[2][4][32];
  __shared__ float sum[LANES ? kNormTeamThreads / 32 * LANES * V * I : 1];
  const int size = LANES ? LANES : blockDim.x;
  const int lane = LANES ? threadIdx.x % LANES : threadIdx.x;
  const int teams = LANES ? kNormTeamThreads / size : 1;
  const long long step = (long long)gridDim.x * teams;
  long long row = (long long)blockIdx.x * teams + (LANES ? threadIdx.x / size : 0);
  const int D = a.D;
  const float inv = 1.f / D;
  const bool layer = a.norm == LA_NORM_LAYER, post = X && a.post_weight;
  const bool bias_grad = a.dbias != nullptr;
  auto both = [](float v) { return CellOf<V>::both(v); };
  auto total = [](C c) { return CellOf<V>::sum(c); };
  int turn = 0;
  Raw<T, V> dy[I], x[I];
  Raw<R, RV> r[I][RN], dr[I][RN];
  auto fetch = [&](long long at) {
    const long long o = at * D;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = (lane + i * size) * V;
      if (c >= D) continue;
      dy[i] = load_raw<T, V>(static_cast<const T *>(a.dy) + o + c);
      if constexpr (X) x[i] = load_raw<T, V>(static_cast<const T *>(a.x) + o + c);
#pragma unroll
      for (int k = 0; k < RN; ++k) {
        r[i][k] = load_raw<R, RV>(static_cast<const R *>(a.r) + o + c + k * RV);
        if (a.dr) dr[i][k] = load_raw<R, RV>(static_cast<const R *>(a.dr) + o + c + k * RV);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < I; ++i) {
    dy[i] = x[i] = Raw<T, V>{};
#pragma unroll
    for (int k = 0; k < RN; ++k) r[i][k] = dr[i][k] = Raw<R, RV>{};
  }
  C w[N], f[N];             // weight; alpha scale post_weight
  C dw[N], db[N], ex[N];    // sums over rows of dy n, dy, e n_x
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int c = (lane + i * size) * V;
    float p[V], s[V];
    params_or<V>(a.weight, c, D, 1.f, p);
    P::pack(p, w + i * H);
    params_or<V>(a.scale, c, D, 1.f, s);
    params_or<V>(X ? a.post_weight : nullptr, c, D, 1.f, p);
#pragma unroll
    for (int e = 0; e < V; ++e) p[e] *= a.alpha * s[e];
    P::pack(p, f + i * H);
  }
#pragma unroll
  for (int j = 0; j < N; ++j) dw[j] = db[j] = ex[j] = C(0);
  if (row < a.rows) fetch(row);
  // A team out of rows stays while another of its warp has one: the sums need
  // the whole warp.
  for (long long first = row - (LANES ? threadIdx.x % 32 / size : 0); first < a.rows;
       first += step, row += step) {
    const bool live = row < a.rows;
    C v[N], g[N], e[N], vx[X ? N : 1];
#pragma unroll
    for (int i = 0; i < I; ++i) {
      float t[V];
      dy[i].unpack(t);
      P::pack(t, g + i * H);
      if constexpr (X) {
        x[i].unpack(t);
        P::pack(t, vx + i * H);
      }
#pragma unroll
      for (int k = 0; k < RN; ++k) r[i][k].unpack(t + k * RV);
      P::pack(t, v + i * H);
#pragma unroll
      for (int k = 0; k < RN; ++k) dr[i][k].unpack(t + k * RV);
      P::pack(t, e + i * H);
    }
    if (row + step < a.rows) fetch(row + step);
    C q0 = C(0), q1 = C(0), q2 = C(0), q3 = C(0);
    float rho, rho_x = 1.f, along, mean_g = 0.f;
    if (layer) {
      C m0 = C(0), m1 = C(0);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        m0 = add2(m0, v[j]);
        if constexpr (X) m1 = add2(m1, vx[j]);
      }
      float m[2] = {total(m0), total(m1)};
      team_sums<LANES>(m, red, turn);
      const C mv = both(-m[0] * inv), mx = both(post ? -m[1] * inv : 0.f);
#pragma unroll
      for (int i = 0; i < I; ++i) {
        const bool in = (lane + i * size) * V < D;
#pragma unroll
        for (int k = 0; k < H; ++k) {
          v[i * H + k] = in ? add2(v[i * H + k], mv) : C(0);
          if constexpr (X) vx[i * H + k] = in ? add2(vx[i * H + k], mx) : C(0);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const C gw = mul2(g[j], w[j]);
      q0 = fma2(v[j], v[j], q0);
      q1 = fma2(gw, v[j], q1);
      if (layer) q2 = add2(gw, q2);
      if constexpr (X) q3 = fma2(vx[j], vx[j], q3);
    }
    if (X || layer) {
      float s[4] = {total(q0), total(q1), total(q2), total(q3)};
      team_sums<LANES>(s, red, turn);
      rho = rsqrtf(fmaf(s[0], inv, a.eps));
      along = s[1];
      if (layer) mean_g = s[2] * inv;
      if (post) rho_x = rsqrtf(fmaf(s[3], inv, a.eps));
    } else {
      float s[2] = {total(q0), total(q1)};
      team_sums<LANES>(s, red, turn);
      rho = rsqrtf(fmaf(s[0], inv, a.eps));
      along = s[1];
    }
    const C rho2 = both(rho), against = both(-along * inv * rho * rho), off = both(-mean_g);
    const C rhox2 = both(rho_x);
    R *dres = static_cast<R *>(a.dresidual) + row * D;
    C x0 = C(0), x1 = C(0);
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = (lane + i * size) * V;
#pragma unroll
      for (int k = 0; k < H; ++k) {
        const int j = i * H + k;
        C t = fma2(g[j], w[j], mul2(against, v[j]));
        if (layer) t = add2(t, off);
        e[j] = fma2(rho2, t, e[j]);
        if (live) {
          dw[j] = fma2(g[j], mul2(v[j], rho2), dw[j]);
          if (bias_grad) db[j] = add2(db[j], g[j]);
        }
      }
      if (live && c < D && a.dresidual) {
        float t[V];
        P::unpack(e + i * H, t);
#pragma unroll
        for (int k = 0; k < RN; ++k) store_vec<R, RV>(dres + c + k * RV, t + k * RV);
      }
#pragma unroll
      for (int k = 0; k < H; ++k) {
        const int j = i * H + k;
        if constexpr (X) {
          vx[j] = mul2(vx[j], rhox2);  // n_x, or x where there is no post norm
          if (live) ex[j] = fma2(e[j], vx[j], ex[j]);
        }
        e[j] = mul2(e[j], f[j]);
        if constexpr (X) {
          x0 = fma2(e[j], vx[j], x0);
          if (layer) x1 = add2(x1, e[j]);
        }
      }
    }
    if constexpr (X) {
      if (post) {
        float xs[2] = {total(x0), total(x1)};
        team_sums<LANES>(xs, red, turn);
        const C along_x = both(-xs[0] * inv), mean = both(layer ? -xs[1] * inv : 0.f);
#pragma unroll
        for (int j = 0; j < N; ++j)
          e[j] = mul2(rhox2, fma2(along_x, vx[j], layer ? add2(e[j], mean) : e[j]));
      }
    }
    T *dx = static_cast<T *>(a.dx) + row * D;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = (lane + i * size) * V;
      float t[V];
      P::unpack(e + i * H, t);
      if (live && c < D) store_vec<T, V>(dx + c, t);
    }
  }
  if (!part) return;
  float *mine = part + (long long)blockIdx.x * D;
  const long long all = (long long)gridDim.x * D;
  // times alpha and, where it is given, a parameter: for the gradients of scale and post_weight
  auto share = [&](const C *acc, float alpha, const float *other) {
    float t[V * I];
#pragma unroll
    for (int i = 0; i < I; ++i) {
      float p[V];
      P::unpack(acc + i * H, t + i * V);
      params_or<V>(other, (lane + i * size) * V, D, 1.f, p);
#pragma unroll
      for (int e = 0; e < V; ++e) t[i * V + e] *= alpha * p[e];
    }
    block_share<V, LANES, I>(t, mine, D, sum);
    mine += all;
  };
  if (a.dweight) share(dw, 1.f, nullptr);
  if (a.dbias) share(db, 1.f, nullptr);
  if constexpr (X) {
    if (a.dpost_weight) share(ex, a.alpha, a.scale);
    if (a.dscale) share(ex, a.alpha, a.post_weight);
  }
}

template <typename T, typename R, int V, bool X>
cudaError_t launch_residual_bwd_v(const ResidualNormBwdArgs &a) {
  return with_bwd_team<V>(a.D, [&](auto lanes, auto items, auto most, int threads) {
    constexpr int LANES = decltype(lanes)::value, I = decltype(items)::value;
    constexpr int MAXT = decltype(most)::value;
    const int teams = LANES ? kNormTeamThreads / LANES : 1;
    const int block = LANES ? kNormTeamThreads : threads;
    const unsigned blocks = norm_bwd_blocks((a.rows + teams - 1) / teams, 512 / block, 1);
    WeightSums w{static_cast<const float *>(a.workspace), (int)blocks, a.D, {}};
    int n = 0;
    for (float *out : {a.dweight, a.dbias, a.dpost_weight, a.dscale})
      if (out) w.out[n++] = out;
    residual_norm_bwd_kernel<T, R, V, LANES, I, X, MAXT><<<blocks, block, 0, a.stream>>>(
        a, n ? static_cast<float *>(a.workspace) : nullptr);
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess || !n ? e : launch_weight_sums(w, n, a.stream);
  });
}

// Rows on 16-byte boundaries, or element by element.
template <typename T, typename R>
cudaError_t launch_residual_bwd(const ResidualNormBwdArgs &a) {
  constexpr int V = Pack16<T>::N;
  bool wide = a.D % V == 0;
  for (const void *p : {a.dy, a.r, a.dr, a.x, static_cast<const void *>(a.dx),
                        static_cast<const void *>(a.dresidual)})
    wide = wide && reinterpret_cast<uintptr_t>(p) % 16 == 0;
  if (a.post_weight || a.dscale)
    return wide ? launch_residual_bwd_v<T, R, V, true>(a) : launch_residual_bwd_v<T, R, 1, true>(a);
  return wide ? launch_residual_bwd_v<T, R, V, false>(a) : launch_residual_bwd_v<T, R, 1, false>(a);
}

// The end of the weights' gradients: a block adds 32 columns, each of its 32 warps
// 128 contiguous bytes of every 32nd row of shares, so that a column's chain of
// additions is short.
constexpr int kSumRows = 32;

__global__ void __launch_bounds__(32 * kSumRows) weight_sum_kernel(const WeightSums w) {
  __shared__ float share[kSumRows][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  const float *p = w.part + (size_t)blockIdx.y * w.parts * w.width + c;
  float s = 0.f;
  if (c < w.width) {
#pragma unroll 4
    for (int i = threadIdx.y; i < w.parts; i += kSumRows) s += p[(size_t)i * w.width];
  }
  share[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  // warp y adds column y's shares
  s = share[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  const int out = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && out < w.width) w.out[blockIdx.y][out] = s;
}

}  // namespace

cudaError_t launch_weight_sums(const WeightSums &w, int count, cudaStream_t stream) {
  weight_sum_kernel<<<dim3((w.width + 31) / 32, count), dim3(32, kSumRows), 0, stream>>>(w);
  return cudaGetLastError();
}

size_t residual_norm_bwd_workspace_bytes(long long rows, int D) {
  return 4 * sizeof(float) * norm_bwd_blocks(rows, kNormMostBlocks, 1) * (size_t)D;
}

cudaError_t launch_residual_norm_bwd(const ResidualNormBwdArgs &a) {
  if (a.dtype == LA_F32) return launch_residual_bwd<float, float>(a);
  return a.res_dtype == LA_F32 ? launch_residual_bwd<__nv_bfloat16, float>(a)
                               : launch_residual_bwd<__nv_bfloat16, __nv_bfloat16>(a);
}

}  // namespace la
