// la_chunk_bwd.cu -- backward pass of chunkwise linear attention: the plan, the
// states between segments, and the decays' gradients from their shares.
#include <algorithm>
#include <cmath>

#include "la_chunk_bwd.cuh"

namespace la {

cudaError_t launch_chunk_bwd_bf16(const ChunkBwd &p, int seqs, bool planes, cudaStream_t stream);
cudaError_t launch_chunk_bwd_tc(const ChunkBwd &p, int seqs, bool planes, cudaStream_t stream);
cudaError_t launch_chunk_bwd_f32(const ChunkBwd &p, int seqs, bool wide, bool bf16,
                                 cudaStream_t stream);

namespace {

constexpr int kMaxPer = 512;  // chunks of a segment (the decays' kernel keeps sums of them)
// Tokens from one kept state to the next, of slow decays: with 1024 the gradients of 2 x 32 x 8192 x
// 128 with per-head decays took 521 us, not 530, and ddecay was up to 7.6e-7 off, not 4.8e-7.
constexpr int kKeep = 512;
constexpr int kShort = 64;    // tokens of the bf16 kernels' one chunk

// How a call runs: which planes, the chunk, the segments.
struct Plan {
  bool tc;      // the tcgen05 kernels
  bool wide;    // padded width 128, else 64
  bool full;    // inputs as three planes
  bool planes;  // states as three planes
  int chunk, chunks, segments, per;
};

// The segments that take the least time on 152 SMs, in units of a chunk of both
// walks: whole waves of blocks, each a segment's chunks and a start; with more than one
// segment also the pass over their own shares, S and G in blocks of their own at 0.2 of a chunk's
// time, and two launches.  Compared when the kernels were up to 4% faster than now (the decays' kept
// states and pairs came later), it picks 2 segments
// for 2 x 32 x 8192 x 128 with decays (517 us; 1: 813, 4: 588, 7: 610), 9 for 1 x 16 x 32768 x 128
// (543; 4: 969, 19: 571), 2 for 4 x 16 x 4096 x 64 (130; 1: 189, 4: 140), 9 for 3 x 5 x 777 x 64 x 128
// fp32 (103; 5: 141, 13: 125), and a chunk each for one sequence of 300 tokens in fp32 (17; 5: 28, 1: 102).
Plan make_plan(const ChunkBwdArgs &a, bool f32_out) {
  Plan p;
  p.wide = std::max(a.dk, a.dv) > 64;
  p.full = a.dtype == LA_F32 || (f32_out && a.phi == LA_PHI_ELU1);
  p.planes = p.full || f32_out;
  // More narrow sequences of up to 64 tokens than there are SMs: tcgen05's block, of which an SM holds
  // one, stands alone with its start, its end and its few products.  64 x 32 x 64 x 64 with token
  // decays 147 us, on tcgen05 197 (elu1 without: 121, 138); 8 x 32 x 64 x 64 28, 31 (elu1 24, 21).  Timed
  // from the host, before: 4 x 32 x 64 x 64 25, 21; 64 x 32 x 96 x 64 276, 256; 64 x 32 x 64 x 128 457, 458
  // (167, 137 without decays).
  p.tc = !p.full && !(a.L <= kShort && !p.wide && (long long)a.B * a.H > 152);
  p.chunk = p.tc ? 128 : p.full ? 32 : kShort;
  p.chunks = (a.L + p.chunk - 1) / p.chunk;
  const long long seqs = (long long)a.B * a.H;
  const long long slots = 152ll * (p.wide || p.tc ? 1 : 3);
  double best = 0;
  p.per = 0;
  for (int per = std::min(p.chunks, kMaxPer); per > 0;) {
    const int n = (p.chunks + per - 1) / per;
    const long long waves = (seqs * n + slots - 1) / slots;
    const long long share_waves = (2 * seqs * (n - 1) + slots - 1) / slots;
    const double cost = waves * (per + 1.5) + (n > 1 ? 0.2 * share_waves * per + 1 : 0);
    if (p.per == 0 || cost < best) best = cost, p.per = per, p.segments = n;
    if ((waves > 4 && n > 1) || per == 1) break;  // finer cuts only add to the work
    per = std::min(per - 1, (p.chunks + n) / (n + 1));  // the longest segments of a finer cut
  }
  return p;
}

size_t round_up(size_t n) { return (n + 255) & ~(size_t)255; }

// The workspace's parts, one behind the other; `base` NULL: their size alone.
size_t lay_out(const ChunkBwdArgs &a, const Plan &plan, bool decay_grad, char *base, ChunkBwd *p,
               float **by_segment) {
  const size_t seqs = (size_t)a.B * a.H, es = (size_t)a.dk * a.dv;
  size_t at = 0;
  auto part = [&](size_t floats) {
    float *r = reinterpret_cast<float *>(base + at);
    at += round_up(floats * sizeof(float));
    return base ? r : nullptr;
  };
  if (a.decay_kind != LA_DECAY_NONE) {
    float *lam = part(2 * seqs * plan.chunks * plan.chunk);
    if (p) p->lam = reinterpret_cast<float2 *>(lam);
  }
  if (plan.segments > 1) {
    float *u = part(seqs * (plan.segments - 1) * es), *w = part(seqs * (plan.segments - 1) * es);
    float *total = part(seqs * plan.segments);
    if (p) p->U = u, p->W = w, p->total = total;
  }
  if (decay_grad) {
    float *rq = part(seqs * a.L), *rk = part(seqs * a.L), *rc = part(seqs * a.L);
    float *cs = plan.tc ? part(seqs * a.L) : nullptr, *rs = plan.tc ? part(seqs * a.L) : nullptr;
    float *around = part(seqs * plan.segments), *sums = part(seqs * plan.segments);
    // Any chunk may hold a strong decay, and then keeps its state.
    const size_t kept = seqs * (plan.chunks - 1), width = plan.wide ? 128 : 64;
    float *states = part(kept * (plan.tc ? width * width : es)), *between = part(kept * kShares);
    float *across = plan.tc ? part(2 * seqs * plan.chunks) : nullptr;
    float *strong = part((seqs * plan.chunks + 3) / 4);
    if (p) {
      p->rq = rq, p->rk = rk, p->rc = rc, p->cs = cs, p->rs = rs, p->around = around;
      p->kept = states, p->between = between, p->across = reinterpret_cast<float2 *>(across);
      p->strong = reinterpret_cast<unsigned char *>(strong);
      *by_segment = sums;
    }
  }
  return at;
}

// The chunks' log2 decays, a warp to a chunk.  The sums are of two floats each: in one, a sum of
// 50 would leave differences of neighbours 4e-6.  A kernel of its own, since the walks would
// wait for these sums chunk by chunk.
__device__ __forceinline__ float2 two_sum(float2 a, float2 b) {
  const float s = a.x + b.x, t = s - a.x;
  const float low = (a.x - (s - t)) + (b.x - t) + (a.y + b.y);  // what s lost, and the low parts
  const float hi = s + low;
  return make_float2(hi, low - (hi - s));
}
__device__ __forceinline__ float2 log2_decay(const ChunkBwd &p, int seq, int t) {
  if (t >= p.L) return make_float2(0.f, 0.f);
  const long long at = (long long)seq * p.L + t;
  float a;
  if (p.decay_kind == LA_DECAY_HEAD) a = p.decay[seq % p.H];
  else if (p.decay_kind == LA_DECAY_TOKEN) a = p.decay[at];
  else a = neg_softplus(p.decay[at]);
  // Below e^-200 a decay counts as e^-200, which is 0 in fp32 in whatever it multiplies; a sum
  // of infinities would be NaN.
  if (a < -200.f) a = -200.f;
  const float hi = a * 1.44269502f;  // log2 e = 1.44269502 + 1.92596299e-8
  return make_float2(hi, fmaf(a, 1.92596299e-8f, fmaf(a, 1.44269502f, -hi)));
}

template <int C>
__global__ void __launch_bounds__(256) chunk_decay_kernel(const ChunkBwd p, int seqs) {
  constexpr int N = C / 32;
  const long long item = (long long)blockIdx.x * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (item >= (long long)seqs * p.chunks) return;
  const int seq = (int)(item / p.chunks), t0 = (int)(item % p.chunks) * C;
  float2 a[N];
  bool strong = false;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    a[i] = log2_decay(p, seq, t0 + lane * N + i);
    strong = strong || a[i].x < kStrong;
  }
  if (p.strong) {
    strong = __any_sync(0xffffffffu, strong);
    if (lane == 0) p.strong[item] = strong;
  }
#pragma unroll
  for (int i = 1; i < N; ++i) a[i] = two_sum(a[i - 1], a[i]);
  float2 run = a[N - 1];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const float2 x = make_float2(__shfl_up_sync(0xffffffffu, run.x, off),
                                 __shfl_up_sync(0xffffffffu, run.y, off));
    if (lane >= off) run = two_sum(x, run);
  }
  float2 before = make_float2(__shfl_up_sync(0xffffffffu, run.x, 1),
                              __shfl_up_sync(0xffffffffu, run.y, 1));
  if (lane == 0) before = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < N; ++i) p.lam[item * C + lane * N + i] = two_sum(before, a[i]);
}

template <int C> cudaError_t launch_chunk_decay(const ChunkBwd &p, int seqs, cudaStream_t stream) {
  const long long blocks = ((long long)seqs * p.chunks + 7) / 8;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  chunk_decay_kernel<C><<<(unsigned)blocks, 256, 0, stream>>>(p, seqs);
  return cudaGetLastError();
}

// U: each segment's own share of S becomes the state behind it; W: its own share of G (of
// segment s + 1 at s) becomes the gradient of the state behind segment s.  Thread: four elements.
__global__ void __launch_bounds__(256) segment_scan_kernel(const ChunkBwd p, int vecs) {
  const int vec = blockIdx.x * 256 + threadIdx.x, seq = blockIdx.y;
  if (vec >= vecs) return;
  const int n = p.segments - 1;
  const bool back = blockIdx.z != 0;
  const float4 *first = reinterpret_cast<const float4 *>(back ? p.dSf : p.S0);
  float4 cur = first ? first[(size_t)seq * vecs + vec] : make_float4(0.f, 0.f, 0.f, 0.f);
  float4 *share = reinterpret_cast<float4 *>(back ? p.W : p.U) + (size_t)seq * n * vecs + vec;
  const float *total = p.total + (size_t)seq * p.segments;
  // Eight segments' loads in flight: the stores behind them may be to the same places.
  for (int i = 0; i < n; i += 8) {
    float4 x[8];
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int s = back ? n - 1 - i - j : i + j;
      if (i + j >= n) continue;
      x[j] = share[(size_t)s * vecs];
      f[j] = total[back ? s + 1 : s];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int s = back ? n - 1 - i - j : i + j;
      if (i + j >= n) continue;
      const float g = ex2_approx(f[j]);
      cur.x = fmaf(g, cur.x, x[j].x), cur.y = fmaf(g, cur.y, x[j].y);
      cur.z = fmaf(g, cur.z, x[j].z), cur.w = fmaf(g, cur.w, x[j].w);
      share[(size_t)s * vecs] = cur;
    }
  }
}

// A block: the tokens of one segment.  Their decays' gradients are sums of pairs (i < t <= j):
//     over s >= t of rq + cs, over s < t of rk + rs, within t's block of BLOCK tokens, rc, and `around`
// the block.  <G, e^L_C S>, the pairs around a chunk, is given for the segment's last chunk and
// where a state was kept; with the chunk's rq it is <G, S> in front of the chunk, and that less the
// next chunk's rk is the next one's.  Around a block of a chunk: those, the chunk's rq behind the block, its rk in front,
// and its pairs across the block.
constexpr int kDecayWarps = 32;

template <int C, int BLOCK>
__global__ void __launch_bounds__(32 * kDecayWarps)
decay_grad_kernel(const ChunkBwd p, float *ddecay, float *by_segment) {
  __shared__ float sum_q[kMaxPer], sum_k[kMaxPer], all[kMaxPer], around_of[kMaxPer];
  __shared__ bool strong[kMaxPer];
  __shared__ double share[kDecayWarps];
  constexpr int N = C / 32, LANES = BLOCK / N, BLOCKS = C / BLOCK;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int seq = blockIdx.x / p.segments, seg = blockIdx.x % p.segments;
  const int c0 = seg * p.per, n = min(p.per, p.chunks - c0);
  const size_t base = (size_t)seq * p.L;
  for (int c = warp; c < n; c += kDecayWarps) {
    float q = 0.f, k = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int t = (c0 + c) * C + lane * N + i;
      if (t < p.L) q += p.rq[base + t], k += p.rk[base + t];
    }
    q = group_sum<32>(q), k = group_sum<32>(k);
    if (lane == 0) {
      sum_q[c] = q, sum_k[c] = k;
      const size_t at = (size_t)seq * p.chunks + c0 + c;
      all[c] = p.lam[at * C + C - 1].x;
      strong[c] = p.strong[at];
    }
  }
  __syncthreads();
  // A thread: the chunks that follow from given sums, and what they are off by at the next
  // one, spread over them: half of what their errors add up to is left.
  auto given = [&](int c) {
    float x = 0.f;
    for (int i = 0; i < kShares; ++i) x += p.between[p.keep_slot(seq, c0 + c) * kShares + i];
    return x;
  };
  for (int x = c0 / p.every + threadIdx.x; x * p.every < c0 + n; x += 32 * kDecayWarps) {
    const int from = max(x * p.every - c0, 0), last = min((x + 1) * p.every - c0, n) - 1;
    float around = last == n - 1 ? p.around[(size_t)seq * p.segments + seg] : given(last);
    int start = last;  // the last chunk whose sum was given
    for (int c = last; c >= from; --c) {
      around_of[c] = around;
      if (c == 0) break;
      around += sum_q[c];
      // Past a decay of 2^-40 nothing of <G, S> is left but the rounding of the sum.
      if (all[c - 1] >= -40.f) around -= sum_k[c - 1];
      else around = 0.f, start = c - 1;
      if (c > from && !strong[c - 1]) continue;
      const float exact = given(c - 1);
      if (start >= c) {
        const float off = (around - exact) / (start - c + 1);
        for (int i = c; i < start; ++i) around_of[i] -= off * (start - i);
      }
      around = exact, start = c - 1;
    }
  }
  __syncthreads();
  double total = 0.0;
  for (int c = warp; c < n; c += kDecayWarps) {
    float q[N], k[N], r[N], cs[N], rs[N];
    float sq = 0.f, sk = 0.f, scs = 0.f, srs = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int t = (c0 + c) * C + lane * N + i;
      const bool live = t < p.L;
      q[i] = live ? p.rq[base + t] : 0.f;
      k[i] = live ? p.rk[base + t] : 0.f;
      r[i] = live ? p.rc[base + t] : 0.f;
      cs[i] = BLOCKS > 1 && live ? p.cs[base + t] : 0.f;
      rs[i] = BLOCKS > 1 && live ? p.rs[base + t] : 0.f;
      sq += q[i], sk += k[i], scs += cs[i], srs += rs[i];
    }
    float around = around_of[c];
    if (BLOCKS > 1) {
      static_assert(BLOCKS == 1 || BLOCKS == 4, "blocks that others lie around: 1 and 2");
      const int block = lane / LANES;
      const float bq = group_sum<LANES>(sq), bk = group_sum<LANES>(sk);
      const float2 across = p.across[(size_t)seq * p.chunks + c0 + c];
#pragma unroll
      for (int x = 0; x < BLOCKS; ++x) {
        const float xq = __shfl_sync(0xffffffffu, bq, x * LANES);
        const float xk = __shfl_sync(0xffffffffu, bk, x * LANES);
        if (x > block) around += xq;
        if (x < block) around += xk;
      }
      around += block == 1 ? across.x : block == 2 ? across.y : 0.f;
    }
    const float q_behind = lanes_sum<false, LANES>(sq + scs, lane);
    const float k_before = lanes_sum<true, LANES>(sk + srs, lane);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int t = (c0 + c) * C + lane * N + i;
      float g = q_behind, before = k_before;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (j >= i) g += q[j] + cs[j];
        if (j < i) before += k[j] + rs[j];
      }
      g += before + r[i] + around;
      if (t >= p.L) continue;
      if (p.decay_kind == LA_DECAY_GATE_LOGIT) g *= -1.f / (1.f + expf(-p.decay[base + t]));
      if (p.decay_kind == LA_DECAY_HEAD) total += g;
      else ddecay[base + t] = g;
    }
  }
  if (p.decay_kind != LA_DECAY_HEAD) return;
  for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
  if (lane == 0) share[warp] = total;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kDecayWarps; ++i) total += share[i];
    by_segment[blockIdx.x] = (float)total;
  }
}

// ddecay[h]: the shares of head h's segments in all sequences, in order.
__global__ void __launch_bounds__(32)
head_decay_kernel(const float *by_segment, float *ddecay, int B, int H, int segments) {
  const int h = blockIdx.x;
  double s = 0.0;
  for (long long i = threadIdx.x; i < (long long)B * segments; i += 32)
    s += by_segment[(i / segments * H + h) * segments + i % segments];
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  if (threadIdx.x == 0) ddecay[h] = (float)s;
}

}  // namespace

cudaError_t launch_segment_scan(const ChunkBwd &p, int seqs, cudaStream_t stream) {
  const int vecs = p.n_k * p.n_v / 4;
  // y: sequences; z: forward, backward
  const int y = std::min(seqs, 32768);
  for (int s = 0; s < seqs; s += y) {
    ChunkBwd part = p;
    const size_t es = (size_t)p.n_k * p.n_v, n = p.segments - 1;
    part.U += s * n * es, part.W += s * n * es, part.total += (size_t)s * p.segments;
    if (part.S0) part.S0 += s * es;
    if (part.dSf) part.dSf += s * es;
    segment_scan_kernel<<<dim3((vecs + 255) / 256, std::min(y, seqs - s), 2), 256, 0, stream>>>(
        part, vecs);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

size_t chunk_bwd_workspace_need(const ChunkBwdArgs &a, bool ddecay, bool dS0) {
  const size_t need = lay_out(a, make_plan(a, ddecay || dS0), ddecay, nullptr, nullptr, nullptr);
  return std::max(need, round_up(1));
}

size_t chunk_bwd_workspace_bytes(const ChunkBwdArgs &a) {
  // Enough for either feature map and any set of outputs.
  size_t most = 0;
  for (int phi : {LA_PHI_IDENTITY, LA_PHI_ELU1})
    for (bool f32_out : {false, true}) {
      ChunkBwdArgs b = a;
      b.phi = phi;
      b.decay_kind = LA_DECAY_TOKEN;
      most = std::max(most, lay_out(b, make_plan(b, f32_out), true, nullptr, nullptr, nullptr));
    }
  return most;
}

cudaError_t launch_chunk_bwd(const ChunkBwdArgs &a) {
  const bool decay_grad = a.ddecay != nullptr, f32_out = decay_grad || a.dS0;
  const Plan plan = make_plan(a, f32_out);
  const long long seqs = (long long)a.B * a.H, blocks = seqs * plan.segments;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  ChunkBwd p{a.q, a.k, a.v, a.dO, a.dq, a.dk_out, a.dv_out, a.decay, a.S0, a.dS_final, a.dS0,
             a.H, a.L, a.dk, a.dv, a.phi, a.decay_kind, plan.chunks, plan.segments, plan.per,
             nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
             nullptr, nullptr, nullptr, kKeep / plan.chunk};
  float *by_segment = nullptr;
  lay_out(a, plan, decay_grad, static_cast<char *>(a.workspace), &p, &by_segment);
  cudaError_t e = cudaSuccess;
  if (a.decay_kind != LA_DECAY_NONE)
    e = plan.chunk == 128  ? launch_chunk_decay<128>(p, (int)seqs, a.stream)
        : plan.chunk == 64 ? launch_chunk_decay<64>(p, (int)seqs, a.stream)
                           : launch_chunk_decay<32>(p, (int)seqs, a.stream);
  if (e != cudaSuccess) return e;
  e = plan.tc ? launch_chunk_bwd_tc(p, (int)seqs, plan.planes, a.stream)
      : plan.full ? launch_chunk_bwd_f32(p, (int)seqs, plan.wide, a.dtype == LA_BF16, a.stream)
                  : launch_chunk_bwd_bf16(p, (int)seqs, plan.planes, a.stream);
  if (e != cudaSuccess || !decay_grad) return e;
  if (plan.chunk == 128)
    decay_grad_kernel<128, 32><<<(unsigned)blocks, 32 * kDecayWarps, 0, a.stream>>>(p, a.ddecay, by_segment);
  else if (plan.chunk == 32)
    decay_grad_kernel<32, 32><<<(unsigned)blocks, 32 * kDecayWarps, 0, a.stream>>>(p, a.ddecay, by_segment);
  else
    decay_grad_kernel<64, 64><<<(unsigned)blocks, 32 * kDecayWarps, 0, a.stream>>>(p, a.ddecay, by_segment);
  if ((e = cudaGetLastError()) != cudaSuccess || a.decay_kind != LA_DECAY_HEAD) return e;
  head_decay_kernel<<<a.H, 32, 0, a.stream>>>(by_segment, a.ddecay, a.B, a.H, plan.segments);
  return cudaGetLastError();
}

}  // namespace la
