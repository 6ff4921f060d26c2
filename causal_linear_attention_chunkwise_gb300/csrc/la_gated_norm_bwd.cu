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
#include <cstdint>

#include "la_block_norm_bwd.cuh"

namespace la {
namespace {

// act(z) and its derivative.
__device__ __forceinline__ void act_and_slope(int act, float z, float &a, float &slope) {
  if (act == LA_ACT_NONE) {
    a = z, slope = 1.f;
    return;
  }
  const float s = sigmoid(z), rest = 1.f - s;
  a = act == LA_ACT_SILU ? z * s : s;
  slope = act == LA_ACT_SILU ? fmaf(a, rest, s) : s * rest;
}

// Weights shared by the heads: the rows are those of all heads, in the order of
// the tokens.  Weights of each head: a block stays with head blockIdx.y.
template <typename T, int V, int LANES, int I, int MAXT>
__global__ void __launch_bounds__(MAXT, LANES ? 2 : 1)
gated_norm_bwd_kernel(const GatedNormBwdArgs a, long long rows, float *part) {
  constexpr int N = V * I;
  __shared__ float red[2][4][32];
  __shared__ float sum[LANES ? kNormTeamThreads / 32 * LANES * N : 1];
  const int size = LANES ? LANES : blockDim.x;
  const int lane = LANES ? threadIdx.x % LANES : threadIdx.x;
  const int teams = LANES ? kNormTeamThreads / size : 1;
  const long long step = (long long)gridDim.x * teams;
  long long r = (long long)blockIdx.x * teams + (LANES ? threadIdx.x / size : 0);
  const int d = a.d, own_head = a.weight_heads > 1 ? blockIdx.y : -1;
  const float inv = 1.f / d;
  const bool gate = a.gate != nullptr, gate_first = gate && a.gate_first;
  const bool layer = a.norm == LA_NORM_LAYER;
  int turn = 0;
  Raw<T, V> x[I], z[I], dy[I];
  struct Place {
    long long bt, x, dx;
    int h;
  };
  auto place = [&](long long row) {
    Place p;
    p.bt = own_head >= 0 ? row : div_index(row, a.H);
    p.h = own_head >= 0 ? own_head : (int)(row - p.bt * a.H);
    const long long b = div_index(p.bt, a.L), t = p.bt - b * a.L;
    p.x = b * a.x_bs + p.h * a.x_hs + t * a.x_ts;
    p.dx = b * a.dx_bs + p.h * a.dx_hs + t * a.dx_ts;
    return p;
  };
  auto fetch = [&](const Place &p) {
    const T *xr = static_cast<const T *>(a.x) + p.x;
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
  float w[N], bias[N], dw[N], db[N];
  const long long w0 = own_head >= 0 ? (long long)own_head * d : 0;
#pragma unroll
  for (int i = 0; i < I; ++i) {
    const int c = (lane + i * size) * V;
    params_or<V>(a.weight ? a.weight + w0 : nullptr, c, d, 1.f, w + i * V);
    params_or<V>(a.bias ? a.bias + w0 : nullptr, c, d, 0.f, bias + i * V);
  }
#pragma unroll
  for (int j = 0; j < N; ++j) dw[j] = db[j] = 0.f;
  Place next{};
  if (r < rows) next = place(r), fetch(next);
  // A team out of rows stays while another of its warp has one: the sums need
  // the whole warp.
  for (long long first = r - (LANES ? threadIdx.x % 32 / size : 0); first < rows;
       first += step, r += step) {
    const bool live = r < rows;
    const Place at = next;
    float v[N], act[N], slope[N], g[N];
#pragma unroll
    for (int i = 0; i < I; ++i) {
      x[i].unpack(v + i * V);
      z[i].unpack(act + i * V);
      dy[i].unpack(g + i * V);
    }
    if (r + step < rows) next = place(r + step), fetch(next);
    if (!live) {
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = act[j] = g[j] = 0.f;
    }
    float keep[N];  // the factor of act's slope: x where the gate comes first, else dy
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (gate) {
        act_and_slope(a.act, act[j], act[j], slope[j]);
      } else {
        act[j] = 1.f, slope[j] = 0.f;
      }
      keep[j] = gate_first ? v[j] : g[j];
      if (gate_first) v[j] *= act[j];
      else g[j] *= act[j];  // the gradient of n w + b
    }
    float mean_g = 0.f;
    float s[3] = {0.f, 0.f, 0.f};
    if (layer) {
      float m[1] = {0.f};
#pragma unroll
      for (int j = 0; j < N; ++j) m[0] += v[j];
      team_sums<LANES>(m, red, turn);
#pragma unroll
      for (int i = 0; i < I; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e)
          v[i * V + e] = (lane + i * size) * V < d ? v[i * V + e] - m[0] * inv : 0.f;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float gw = g[j] * w[j];
      s[0] = fmaf(v[j], v[j], s[0]);
      s[1] = fmaf(gw, v[j], s[1]);
      s[2] += gw;
    }
    team_sums<LANES>(s, red, turn);
    const float rs = rsqrtf(fmaf(s[0], inv, a.eps));
    if (layer) mean_g = s[2] * inv;
    const float along = s[1] * inv * rs * rs;  // mean(g n) r, for n = v r
    T *dxr = static_cast<T *>(a.dx) + at.dx;
    T *dzr = static_cast<T *>(a.dgate) + at.bt * a.dgate_stride + (long long)at.h * d;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int c = (lane + i * size) * V;
      float ox[V], oz[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int j = i * V + e;
        const float n = v[j] * rs;
        const float u = rs * (fmaf(g[j], w[j], -mean_g) - along * v[j]);
        if (live) {
          dw[j] = fmaf(g[j], n, dw[j]);
          db[j] += g[j];
        }
        ox[e] = gate_first ? u * act[j] : u;
        oz[e] = (gate_first ? u : fmaf(n, w[j], bias[j])) * keep[j] * slope[j];
      }
      if (!live || c >= d) continue;
      store_vec<T, V>(dxr + c, ox);
      if (gate) store_vec<T, V>(dzr + c, oz);
    }
  }
  if (!part) return;
  const long long width = (long long)a.weight_heads * d;
  float *mine = part + (long long)blockIdx.x * width + w0;
  if (a.dweight) {
    block_share<V, LANES, I>(dw, mine, d, sum);
    mine += (long long)gridDim.x * width;
  }
  if (a.dbias) block_share<V, LANES, I>(db, mine, d, sum);
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
    const unsigned blocks = norm_bwd_blocks((rows + teams - 1) / teams, block, heads);
    float *part = sums ? static_cast<float *>(a.workspace) : nullptr;
    gated_norm_bwd_kernel<T, V, LANES, I, MAXT>
        <<<dim3(blocks, heads), block, 0, a.stream>>>(a, rows, part);
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
  return 2 * sizeof(float) * norm_bwd_blocks(rows, 1, heads) * (size_t)weight_heads * d;
}

cudaError_t launch_gated_norm_bwd(const GatedNormBwdArgs &a) {
  return a.dtype == LA_F32 ? launch_t<float>(a) : launch_t<__nv_bfloat16>(a);
}

}  // namespace la
