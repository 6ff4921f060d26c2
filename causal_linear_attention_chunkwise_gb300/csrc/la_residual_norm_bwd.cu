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
// alone.  r is read as the forward pass stored it.
#include <cstdint>

#include "la_block_norm_bwd.cuh"

namespace la {
namespace {

// X: x is read (a post norm, or a scale's gradient).
template <typename T, typename R, int V, int LANES, int I, bool X, int MAXT>
__global__ void __launch_bounds__(MAXT, LANES ? 2 : 1)
residual_norm_bwd_kernel(const ResidualNormBwdArgs a, float *part) {
  constexpr int N = V * I, RV = V < Pack16<R>::N ? V : Pack16<R>::N, RN = V / RV;
  __shared__ float red[2][4][32];
  __shared__ float sum[LANES ? kNormTeamThreads / 32 * LANES * N : 1];
  const int size = LANES ? LANES : blockDim.x;
  const int lane = LANES ? threadIdx.x % LANES : threadIdx.x;
  const int teams = LANES ? kNormTeamThreads / size : 1;
  const long long step = (long long)gridDim.x * teams;
  long long row = (long long)blockIdx.x * teams + (LANES ? threadIdx.x / size : 0);
  const int D = a.D;
  const float inv = 1.f / D;
  const bool layer = a.norm == LA_NORM_LAYER, post = X && a.post_weight;
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
  float w[N], s[N], p[N];  // weight, alpha scale, post_weight
  float dw[N], db[N], ds[N], dp[N];
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int c = (lane + i * size) * V;
    params_or<V>(a.weight, c, D, 1.f, w + i * V);
    params_or<V>(a.scale, c, D, 1.f, s + i * V);
    params_or<V>(X ? a.post_weight : nullptr, c, D, 1.f, p + i * V);
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    s[j] *= a.alpha;
    dw[j] = db[j] = ds[j] = dp[j] = 0.f;
  }
  if (row < a.rows) fetch(row);
  // A team out of rows stays while another of its warp has one: the sums need
  // the whole warp.
  for (long long first = row - (LANES ? threadIdx.x % 32 / size : 0); first < a.rows;
       first += step, row += step) {
    const bool live = row < a.rows;
    float v[N], g[N], e[N], vx[N];
#pragma unroll
    for (int i = 0; i < I; ++i) {
      dy[i].unpack(g + i * V);
      x[i].unpack(vx + i * V);
#pragma unroll
      for (int k = 0; k < RN; ++k) {
        r[i][k].unpack(v + i * V + k * RV);
        dr[i][k].unpack(e + i * V + k * RV);
      }
    }
    if (row + step < a.rows) fetch(row + step);
    float sums[4] = {0.f, 0.f, 0.f, 0.f};
    float mean_x = 0.f;
    if (layer) {
      float m[2] = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < N; ++j) m[0] += v[j], m[1] += vx[j];
      team_sums<LANES>(m, red, turn);
      mean_x = post ? m[1] * inv : 0.f;
#pragma unroll
      for (int i = 0; i < I; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const bool in = (lane + i * size) * V < D;
          v[i * V + k] = in ? v[i * V + k] - m[0] * inv : 0.f;
          if (post) vx[i * V + k] = in ? vx[i * V + k] - mean_x : 0.f;
        }
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float gw = g[j] * w[j];
      sums[0] = fmaf(v[j], v[j], sums[0]);
      sums[1] = fmaf(gw, v[j], sums[1]);
      sums[2] += gw;
      sums[3] = fmaf(vx[j], vx[j], sums[3]);
    }
    team_sums<LANES>(sums, red, turn);
    const float rho = rsqrtf(fmaf(sums[0], inv, a.eps));
    const float mean_g = layer ? sums[2] * inv : 0.f, along = sums[1] * inv * rho * rho;
    const float rho_x = post ? rsqrtf(fmaf(sums[3], inv, a.eps)) : 1.f;
    R *dres = static_cast<R *>(a.dresidual) + row * D;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = (lane + i * size) * V;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int j = i * V + k;
        e[j] = fmaf(rho, fmaf(g[j], w[j], -mean_g) - along * v[j], e[j]);
        if (live) {
          dw[j] = fmaf(g[j], v[j] * rho, dw[j]);
          db[j] += g[j];
        }
      }
      if (!live || c >= D || !a.dresidual) continue;
#pragma unroll
      for (int k = 0; k < RN; ++k) store_vec<R, RV>(dres + c + k * RV, e + i * V + k * RV);
    }
    float xs[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if constexpr (X) {
        vx[j] *= rho_x;  // n_x, or x where there is no post norm
        if (live) {
          ds[j] = fmaf(a.alpha * e[j], vx[j] * p[j], ds[j]);
          dp[j] = fmaf(s[j] * e[j], vx[j], dp[j]);
        }
      }
      e[j] *= s[j] * p[j];
      if constexpr (X) {
        xs[0] = fmaf(e[j], vx[j], xs[0]);
        xs[1] += e[j];
      }
    }
    if (post) {
      team_sums<LANES>(xs, red, turn);
      const float along_x = xs[0] * inv, mean = layer ? xs[1] * inv : 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j) e[j] = rho_x * (e[j] - mean - along_x * vx[j]);
    }
    T *dx = static_cast<T *>(a.dx) + row * D;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = (lane + i * size) * V;
      if (live && c < D) store_vec<T, V>(dx + c, e + i * V);
    }
  }
  if (!part) return;
  float *mine = part + (long long)blockIdx.x * D;
  const long long all = (long long)gridDim.x * D;
  if (a.dweight) block_share<V, LANES, I>(dw, mine, D, sum), mine += all;
  if (a.dbias) block_share<V, LANES, I>(db, mine, D, sum), mine += all;
  if constexpr (X) {
    if (a.dpost_weight) block_share<V, LANES, I>(dp, mine, D, sum), mine += all;
    if (a.dscale) block_share<V, LANES, I>(ds, mine, D, sum);
  }
}

template <typename T, typename R, int V, bool X>
cudaError_t launch_residual_bwd_v(const ResidualNormBwdArgs &a) {
  return with_bwd_team<V>(a.D, [&](auto lanes, auto items, auto most, int threads) {
    constexpr int LANES = decltype(lanes)::value, I = decltype(items)::value;
    constexpr int MAXT = decltype(most)::value;
    const int teams = LANES ? kNormTeamThreads / LANES : 1;
    const int block = LANES ? kNormTeamThreads : threads;
    const unsigned blocks = norm_bwd_blocks((a.rows + teams - 1) / teams, block, 1);
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
  return 4 * sizeof(float) * norm_bwd_blocks(rows, 1, 1) * (size_t)D;
}

cudaError_t launch_residual_norm_bwd(const ResidualNormBwdArgs &a) {
  if (a.dtype == LA_F32) return launch_residual_bwd<float, float>(a);
  return a.res_dtype == LA_F32 ? launch_residual_bwd<__nv_bfloat16, float>(a)
                               : launch_residual_bwd<__nv_bfloat16, __nv_bfloat16>(a);
}

}  // namespace la
