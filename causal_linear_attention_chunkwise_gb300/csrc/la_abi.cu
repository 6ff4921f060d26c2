// la_abi.cu -- the extern "C" boundary: argument validation, dispatch to the
// kernel launchers, the process-wide feature map, error reporting.
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "../../include/la_gb300.h"
#include "la_common.cuh"
#include "la_internal.h"

namespace la {

__device__ unsigned int g_device_error;

namespace {
std::atomic<int> g_phi{LA_PHI_IDENTITY};
thread_local char g_msg[512] = "";

la_status fail(la_status s, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof g_msg, fmt, ap);
  va_end(ap);
  return s;
}

la_status ok() {
  g_msg[0] = '\0';
  return LA_OK;
}

la_status cuda_fail(cudaError_t e, const char *where) {
  return fail(LA_ERR_CUDA, "%s: %s (%s)", where, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

bool supported_d(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

// Copy `src` to `dst` (or zero `dst` when src is null): the state after no tokens.
cudaError_t pass_through_state(float *dst, const float *src, size_t bytes, cudaStream_t st) {
  if (!dst) return cudaSuccess;
  if (!src) return cudaMemsetAsync(dst, 0, bytes, st);
  if (src == dst) return cudaSuccess;
  return cudaMemcpyAsync(dst, src, bytes, cudaMemcpyDeviceToDevice, st);
}

// Checks shared by la_normalised_fwd, la_channel_gate_fwd and la_delta_fwd.
// Returns LA_OK with *done = false when the kernel is to run; otherwise the
// call ends with the returned status (LA_OK with *done = true: an empty batch,
// or L = 0 with the states passed through).
la_status check_variant(const char *fn, const void *q, const void *k, const void *v, int dtype,
                        int B, int H, int L, int d_k, int d_v, int chunk, bool uses_chunk,
                        const float *S0, const float *z0, void *O, float *S_final,
                        float *z_final, cudaStream_t st, bool *done) {
  *done = true;
  if (dtype != LA_F32 && dtype != LA_BF16)
    return fail(LA_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, dtype);
  if (B < 0 || H < 0 || L < 0 || d_k <= 0 || d_v <= 0 || (uses_chunk && chunk <= 0))
    return fail(LA_ERR_INVALID_ARG, "%s: bad sizes B=%d H=%d L=%d d_k=%d d_v=%d chunk=%d", fn,
                B, H, L, d_k, d_v, chunk);
  if (!supported_d(d_k) || !supported_d(d_v))
    return fail(LA_ERR_UNSUPPORTED, "%s: d_k=%d d_v=%d not in {16,32,64,128}", fn, d_k, d_v);
  if (uses_chunk && chunk > 64)
    return fail(LA_ERR_UNSUPPORTED, "%s: chunk %d > 64 is not supported", fn, chunk);
  if ((size_t)B * H == 0) return ok();
  if ((S0 && !aligned16(S0)) || (S_final && !aligned16(S_final)) || (z0 && !aligned16(z0)) ||
      (z_final && !aligned16(z_final)))
    return fail(LA_ERR_INVALID_ARG, "%s: state pointers must be 16-byte aligned", fn);
  if (L == 0) {
    const size_t sb = (size_t)B * H * d_k * d_v * sizeof(float);
    const size_t zb = (size_t)B * H * d_k * sizeof(float);
    cudaError_t e = pass_through_state(S_final, S0, sb, st);
    if (e == cudaSuccess) e = pass_through_state(z_final, z0, zb, st);
    if (e != cudaSuccess) return cuda_fail(e, fn);
    return ok();
  }
  if (!q || !k || !v || !O)
    return fail(LA_ERR_INVALID_ARG, "%s: q, k, v and O must be non-null", fn);
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(O))
    return fail(LA_ERR_INVALID_ARG, "%s: tensors must start on a 16-byte boundary", fn);
  *done = false;
  return ok();
}

la_status run_variant(const char *fn, const VariantArgs &a) {
  cudaError_t e = launch_variant(a);
  if (e != cudaSuccess) return cuda_fail(e, fn);
  return ok();
}

// Tokens and channels of the calls whose kernels add a tile to them in 32 bits.
constexpr int kMaxLen = 1 << 30;

// The bytes that `rows` rows of `width` elements, `stride` elements apart, lie in.
struct Rows {
  const void *p;
  long long rows, width, stride;
  size_t elt;
};

// Whether an output shares an element with an input.  Rows of equal pitch may
// interleave (two slices of one wider tensor).
bool overlap(const Rows &a, const Rows &b) {
  if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  const uintptr_t a1 = a0 + ((size_t)(a.rows - 1) * a.stride + a.width) * a.elt;
  const uintptr_t b1 = b0 + ((size_t)(b.rows - 1) * b.stride + b.width) * b.elt;
  if (a1 <= b0 || b1 <= a0) return false;
  const uintptr_t pitch = (uintptr_t)a.stride * a.elt;
  if (pitch != (uintptr_t)b.stride * b.elt || pitch == 0) return true;
  const uintptr_t ahead = b0 >= a0 ? (b0 - a0) % pitch : (pitch - (a0 - b0) % pitch) % pitch;
  return ahead < a.width * a.elt || ahead + b.width * b.elt > pitch;
}

// The same for dense ranges of bytes.
Rows dense(const void *p, size_t bytes) { return {p, 1, (long long)bytes, (long long)bytes, 1}; }

// n fp32 parameters or int32 lengths.
Rows params(const void *p, long long n) { return dense(p, (size_t)n * 4); }

// Whether an output shares an element with one of several inputs.
template <size_t N>
bool overlap_any(const Rows &out, const Rows (&in)[N]) {
  for (const Rows &r : in)
    if (overlap(out, r)) return true;
  return false;
}

bool aligned_elt(const void *p, size_t elt) {
  return (reinterpret_cast<uintptr_t>(p) & (elt - 1)) == 0;
}

// Sizes that la_chunk_bwd supports, with tokens to work on.
bool chunk_bwd_sizes(int B, int H, int L, int d_k, int d_v, int chunk, int dtype) {
  return B > 0 && H > 0 && L > 0 && L <= kMaxLen && (long long)B * H <= 0x7fffffffll &&
         supported_d(d_k) && supported_d(d_v) && chunk >= 1 && chunk <= 64 &&
         (dtype == LA_F32 || dtype == LA_BF16);
}

// A [B,H,L,d] tensor with strides, in elements; its last axis is dense.
struct Heads {
  const void *p;
  long long n[3], s[3];  // b, h, t
  int d;
  size_t elt;
};
Heads heads_of(const void *p, int B, int H, int L, int d, long long bs, long long hs,
               long long ts, size_t elt) {
  return {p, {B, H, L}, {bs, hs, ts}, d, elt};
}
// [B,L,H*d] rows `stride` elements apart, seen as such a tensor.
Heads token_rows(const void *p, int B, int H, int L, int d, long long stride, size_t elt) {
  return heads_of(p, B, H, L, d, L * stride, d, stride, elt);
}
// All that it spans, as one row.
Rows span_of(const Heads &x) {
  long long span = x.d;
  for (int i = 0; i < 3; ++i) span += (x.n[i] - 1) * x.s[i];
  return {x.p, 1, span, span, x.elt};
}

// One axis of the differences between two tensors' indices: lo .. hi times s.
struct Axis {
  long long s, lo, hi;
};
// Whether `delta` is a sum of multiples of the axes' strides, the largest first, and one of
// lo .. hi.  Where a stride is shorter than what lies inside it there may be many ways to try:
// they count as one that fits.
bool reaches(const Axis *axis, int axes, long long lo, long long hi, long long delta) {
  if (axes == 0) return lo <= delta && delta <= hi;
  long long least = lo, most = hi;  // of what the axes inside this one add
  for (int i = 1; i < axes; ++i) least += axis[i].lo * axis[i].s, most += axis[i].hi * axis[i].s;
  const long long s = axis->s;
  auto floor_div = [&](long long x) { return x / s - (x % s < 0); };
  const long long first = -floor_div(most - delta), last = floor_div(delta - least);
  const long long from = first > axis->lo ? first : axis->lo, to = last < axis->hi ? last : axis->hi;
  if (to - from > 3) return true;
  for (long long k = from; k <= to; ++k)
    if (reaches(axis + 1, axes - 1, lo, hi, delta - k * s)) return true;
  return false;
}

// Whether two such tensors share an element.  Tensors of one set of strides may interleave in any
// way (slices of a packed projection, whatever the order of its axes, or of a longer batch); those
// of unlike strides must not lie in one range.
bool overlap(const Heads &a, const Heads &b) {
  if (!a.p || !b.p) return false;
  if (!overlap(span_of(a), span_of(b))) return false;
  Axis axis[3];
  int axes = 0;
  for (int i = 0; i < 3; ++i) {
    if (a.n[i] > 1 && b.n[i] > 1 && a.s[i] != b.s[i]) return true;
    const long long s = a.n[i] > 1 ? a.s[i] : b.s[i];
    if ((a.n[i] == 1 && b.n[i] == 1) || s == 0) continue;
    int at = axes++;
    for (; at > 0 && axis[at - 1].s < s; --at) axis[at] = axis[at - 1];
    axis[at] = {s, 1 - b.n[i], a.n[i] - 1};
  }
  const long long bytes = (long long)(reinterpret_cast<uintptr_t>(b.p) -
                                      reinterpret_cast<uintptr_t>(a.p));
  return reaches(axis, axes, 1 - b.d, a.d - 1, bytes / (long long)a.elt);
}

// Whether no two elements of a [B,H,L,d] tensor lie in one place, as an output's may not.
bool own_places(int B, int H, int L, int d, long long bs, long long hs, long long ts) {
  long long n[3] = {B, H, L}, s[3] = {bs, hs, ts}, extent = d;
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (s[j] < s[i]) {
        const long long a = s[i], b = n[i];
        s[i] = s[j], n[i] = n[j], s[j] = a, n[j] = b;
      }
  for (int i = 0; i < 3; ++i) {
    if (n[i] == 1) continue;
    if (s[i] < extent) return false;
    extent += (n[i] - 1) * s[i];
  }
  return true;
}

la_status rotary(const char *fn, RotaryArgs a) {
  if (a.dtype != LA_F32 && a.dtype != LA_BF16)
    return fail(LA_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, a.dtype);
  if (a.B < 0 || a.heads_q < 0 || a.heads_k < 0 || a.L < 0 || a.d <= 0)
    return fail(LA_ERR_INVALID_ARG, "%s: bad sizes B=%d heads=%d, %d L=%d d=%d", fn, a.B,
                a.heads_q, a.heads_k, a.L, a.d);
  if (a.rot < 2 || a.rot > a.d || a.rot % 2)
    return fail(LA_ERR_INVALID_ARG, "%s: rotary_dim=%d is no even number in 2..d=%d", fn, a.rot,
                a.d);
  if (a.d > 16384 || a.heads_q > 16384 || a.heads_k > 16384 || a.L > kMaxLen)
    return fail(LA_ERR_UNSUPPORTED,
                "%s: d=%d or heads=%d, %d above 16384, or L=%d above 2^30", fn, a.d, a.heads_q,
                a.heads_k, a.L);
  if (!a.k.p && !a.k_out.p) a.heads_k = 0;
  if (a.B == 0 || a.L == 0 || a.heads_q + a.heads_k == 0) return ok();
  const size_t elt = a.dtype == LA_F32 ? 4 : 2;
  Heads in[2], out[2];
  const RotaryTensor x[] = {a.q, a.k}, y[] = {a.q_out, a.k_out};
  const int heads[] = {a.heads_q, a.heads_k};
  for (int i = 0; i < 2; ++i) {
    if (heads[i] == 0) {
      in[i] = out[i] = Heads{nullptr, {}, {}, 0, elt};
      continue;
    }
    if (!x[i].p || !y[i].p)
      return fail(LA_ERR_INVALID_ARG, "%s: q, q_out, or one of k and k_out, is null", fn);
    if (!aligned_elt(x[i].p, elt) || !aligned_elt(y[i].p, elt))
      return fail(LA_ERR_INVALID_ARG, "%s: pointers must be aligned to their elements", fn);
    for (const RotaryTensor *t : {&x[i], &y[i]})
      if (t->bs < 0 || t->hs < 0 || t->ts < 0)
        return fail(LA_ERR_INVALID_ARG, "%s: negative stride", fn);
    if (!own_places(a.B, heads[i], a.L, a.d, y[i].bs, y[i].hs, y[i].ts))
      return fail(LA_ERR_INVALID_ARG, "%s: an output's strides put two elements in one place", fn);
    in[i] = heads_of(x[i].p, a.B, heads[i], a.L, a.d, x[i].bs, x[i].hs, x[i].ts, elt);
    out[i] = heads_of(y[i].p, a.B, heads[i], a.L, a.d, y[i].bs, y[i].hs, y[i].ts, elt);
  }
  if (!a.inv_freq) return fail(LA_ERR_INVALID_ARG, "%s: inv_freq must be non-null", fn);
  for (const void *p : {static_cast<const void *>(a.inv_freq),
                        static_cast<const void *>(a.positions),
                        static_cast<const void *>(a.offsets),
                        static_cast<const void *>(a.lengths)})
    if (!aligned_elt(p, 4))
      return fail(LA_ERR_INVALID_ARG, "%s: inv_freq, positions, offsets and lengths must be "
                  "4-byte aligned", fn);
  const Rows par[] = {params(a.inv_freq, a.rot / 2), params(a.positions, (long long)a.B * a.L),
                      params(a.offsets, a.B), params(a.lengths, a.B)};
  for (int i = 0; i < 2; ++i) {
    const bool in_place = x[i].p == y[i].p && (a.B == 1 || x[i].bs == y[i].bs) &&
                          (heads[i] == 1 || x[i].hs == y[i].hs) &&
                          (a.L == 1 || x[i].ts == y[i].ts);
    if ((!in_place && overlap(out[i], in[i])) || overlap(out[i], in[1 - i]))
      return fail(LA_ERR_INVALID_ARG, "%s: an output overlaps an input", fn);
  }
  if (overlap(out[0], out[1]))
    return fail(LA_ERR_INVALID_ARG, "%s: q_out and k_out overlap", fn);
  for (const Heads &o : out)
    if (overlap_any(span_of(o), par))
      return fail(LA_ERR_INVALID_ARG,
                  "%s: an output overlaps inv_freq, positions, offsets or lengths", fn);
  cudaError_t e = launch_rotary(a);
  if (e != cudaSuccess) return cuda_fail(e, fn);
  return ok();
}

const char *kernel_name(unsigned int id) {
  switch (id) {
    case KID_PREFILL_TC_STATE: return "prefill segment-state kernel";
    case KID_PREFILL_TC_OUT: return "prefill chunk-output kernel";
    case KID_SELFTEST: return "wait-timeout self-test kernel";
    case KID_NONCAUSAL: return "non-causal output kernel";
    case KID_CHANNEL_GATE_TC: return "per-channel gate tensor-core kernel";
    case KID_DELTA_TC: return "delta-rule tensor-core kernel";
    case KID_CHUNK_BWD_TC: return "attention backward tensor-core kernel";
    default: return "unknown kernel";
  }
}
}  // namespace

void set_last_error(const char *msg) { snprintf(g_msg, sizeof g_msg, "%s", msg); }

unsigned int *device_error_word() {
  // The symbol's device address, looked up for the current device on each
  // call (cheap; avoids caching an address across devices).
  void *p = nullptr;
  if (cudaGetSymbolAddress(&p, g_device_error) != cudaSuccess) {
    cudaGetLastError();
    return nullptr;
  }
  return static_cast<unsigned int *>(p);
}

}  // namespace la

using namespace la;

extern "C" {

la_status la_set_feature_map(int phi) {
  if (phi != LA_PHI_IDENTITY && phi != LA_PHI_ELU1)
    return fail(LA_ERR_INVALID_ARG, "la_set_feature_map: unknown feature map %d", phi);
  g_phi.store(phi);
  return ok();
}

int la_get_feature_map(void) { return g_phi.load(); }

size_t la_chunk_fwd_workspace_bytes(int B, int H, int L, int d_k, int d_v, int chunk, int dtype) {
  PrefillArgs a{};
  a.dtype = dtype; a.B = B; a.H = H; a.L = L; a.dk = d_k; a.dv = d_v; a.chunk = chunk;
  if (B <= 0 || H <= 0 || L <= 0) return 0;
  if (prefill_tc_supported(a)) return prefill_tc_workspace_bytes(B, H, L, d_k);
  return 0;
}

int la_chunk_fwd_kernel_count(int B, int H, int L, int d_k, int d_v, int chunk, int dtype) {
  if (B <= 0 || H <= 0 || L <= 0) return 0;
  if ((dtype != LA_F32 && dtype != LA_BF16) || !supported_d(d_k) || !supported_d(d_v) ||
      chunk < 1 || chunk > 64)
    return 0;
  PrefillArgs a{};
  a.dtype = dtype; a.B = B; a.H = H; a.L = L; a.dk = d_k; a.dv = d_v; a.chunk = chunk;
  if (prefill_tc_supported(a)) return prefill_tc_kernel_count(B, H, L, d_k);
  return 1;
}

la_status la_chunk_fwd(const void *q, const void *k, const void *v, int dtype, int B, int H,
                       int L, int d_k, int d_v, int chunk, int decay_kind, const float *decay,
                       const float *S0, void *O, float *S_final, void *workspace,
                       size_t ws_bytes, void *cuda_stream) {
  if (dtype != LA_F32 && dtype != LA_BF16)
    return fail(LA_ERR_INVALID_ARG, "la_chunk_fwd: unknown dtype %d", dtype);
  if (B < 0 || H < 0 || L < 0 || d_k <= 0 || d_v <= 0 || chunk <= 0)
    return fail(LA_ERR_INVALID_ARG,
                "la_chunk_fwd: bad sizes B=%d H=%d L=%d d_k=%d d_v=%d chunk=%d", B, H, L, d_k,
                d_v, chunk);
  if (decay_kind < LA_DECAY_NONE || decay_kind > LA_DECAY_GATE_LOGIT)
    return fail(LA_ERR_INVALID_ARG, "la_chunk_fwd: unknown decay kind %d", decay_kind);
  if (!supported_d(d_k) || !supported_d(d_v))
    return fail(LA_ERR_UNSUPPORTED, "la_chunk_fwd: d_k=%d d_v=%d not in {16,32,64,128}", d_k,
                d_v);
  if (chunk > 64)
    return fail(LA_ERR_UNSUPPORTED, "la_chunk_fwd: chunk %d > 64 is not supported", chunk);
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const size_t state_bytes = (size_t)B * H * d_k * d_v * sizeof(float);
  if ((size_t)B * H == 0) return ok();
  if (L == 0) {  // nothing to attend to: the final state is the initial one
    if (!S_final) return ok();
    if (!aligned16(S_final) || (S0 && !aligned16(S0)))
      return fail(LA_ERR_INVALID_ARG, "la_chunk_fwd: state pointers must be 16-byte aligned");
    cudaError_t e = S0 ? (S0 == S_final ? cudaSuccess
                                        : cudaMemcpyAsync(S_final, S0, state_bytes,
                                                          cudaMemcpyDeviceToDevice, st))
                       : cudaMemsetAsync(S_final, 0, state_bytes, st);
    if (e != cudaSuccess) return cuda_fail(e, "la_chunk_fwd (L=0)");
    return ok();
  }
  if (!q || !k || !v || !O)
    return fail(LA_ERR_INVALID_ARG, "la_chunk_fwd: q, k, v and O must be non-null");
  if (decay_kind != LA_DECAY_NONE && !decay)
    return fail(LA_ERR_INVALID_ARG, "la_chunk_fwd: decay kind %d needs a decay pointer",
                decay_kind);
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(O) ||
      (S0 && !aligned16(S0)) || (S_final && !aligned16(S_final)))
    return fail(LA_ERR_INVALID_ARG, "la_chunk_fwd: tensors must start on a 16-byte boundary");

  PrefillArgs a{q, k, v, dtype, B, H, L, d_k, d_v, chunk, g_phi.load(), decay_kind,
                decay_kind == LA_DECAY_NONE ? nullptr : decay, S0, O, S_final,
                workspace, ws_bytes, st};
  if (prefill_tc_supported(a)) {
    size_t need = prefill_tc_workspace_bytes(B, H, L, d_k);
    if (need > 0 && (!workspace || ws_bytes < need))
      return fail(LA_ERR_INVALID_ARG,
                  "la_chunk_fwd: workspace of %zu bytes needed, %zu given", need,
                  workspace ? ws_bytes : (size_t)0);
    if (need > 0 && !aligned16(workspace))
      return fail(LA_ERR_INVALID_ARG, "la_chunk_fwd: workspace must be 16-byte aligned");
    const char *why = nullptr;
    cudaError_t e = launch_prefill_tc(a, &why);
    if (e != cudaSuccess) return cuda_fail(e, why ? why : "la_chunk_fwd (tcgen05 path)");
    return ok();
  }
  cudaError_t e = launch_prefill_simt(a);
  if (e != cudaSuccess) return cuda_fail(e, "la_chunk_fwd (SIMT path)");
  return ok();
}

size_t la_noncausal_fwd_workspace_bytes(int B, int H, int L, int d_k, int d_v) {
  if (d_k != d_v || (d_k != 64 && d_k != 128)) return 0;
  return noncausal_workspace_bytes(B, H, L, d_k);
}

la_status la_noncausal_fwd(const void *q, const void *k, const void *v, int dtype, int B, int H,
                           int L, int d_k, int d_v, void *O, float *S, void *workspace,
                           size_t ws_bytes, void *cuda_stream) {
  if (dtype != LA_F32 && dtype != LA_BF16)
    return fail(LA_ERR_INVALID_ARG, "la_noncausal_fwd: unknown dtype %d", dtype);
  if (B < 0 || H < 0 || L < 0 || d_k <= 0 || d_v <= 0)
    return fail(LA_ERR_INVALID_ARG, "la_noncausal_fwd: bad sizes B=%d H=%d L=%d d_k=%d d_v=%d",
                B, H, L, d_k, d_v);
  if (dtype != LA_BF16 || d_k != d_v || (d_k != 64 && d_k != 128))
    return fail(LA_ERR_UNSUPPORTED,
                "la_noncausal_fwd: needs bf16 with d_k = d_v in {64, 128} (dtype %d, %d x %d)",
                dtype, d_k, d_v);
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if ((size_t)B * H == 0) return ok();
  if (S && !aligned16(S))
    return fail(LA_ERR_INVALID_ARG, "la_noncausal_fwd: S must start on a 16-byte boundary");
  if (L == 0) {  // no tokens: the state is zero and there is no output
    if (S) {
      cudaError_t e = cudaMemsetAsync(S, 0, (size_t)B * H * d_k * d_v * sizeof(float), st);
      if (e != cudaSuccess) return cuda_fail(e, "la_noncausal_fwd (L=0)");
    }
    return ok();
  }
  if (!q || !k || !v || !O)
    return fail(LA_ERR_INVALID_ARG, "la_noncausal_fwd: q, k, v and O must be non-null");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(O))
    return fail(LA_ERR_INVALID_ARG, "la_noncausal_fwd: tensors must start on a 16-byte boundary");
  const size_t need = noncausal_workspace_bytes(B, H, L, d_k);
  if (!workspace || ws_bytes < need)
    return fail(LA_ERR_INVALID_ARG, "la_noncausal_fwd: workspace of %zu bytes needed, %zu given",
                need, workspace ? ws_bytes : (size_t)0);
  if (!aligned16(workspace))
    return fail(LA_ERR_INVALID_ARG, "la_noncausal_fwd: workspace must be 16-byte aligned");
  NoncausalArgs a{q, k, v, B, H, L, d_k, g_phi.load(), O, S, workspace, ws_bytes, st};
  const char *why = nullptr;
  cudaError_t e = launch_noncausal(a, &why);
  if (e != cudaSuccess) return cuda_fail(e, why ? why : "la_noncausal_fwd");
  return ok();
}

la_status la_decode_step(const void *q, const void *k, const void *v, int dtype, int B, int H,
                         int d_k, int d_v, const float *log_alpha, float *S, void *o,
                         void *cuda_stream) {
  if (dtype != LA_F32 && dtype != LA_BF16)
    return fail(LA_ERR_INVALID_ARG, "la_decode_step: unknown dtype %d", dtype);
  if (B < 0 || H < 0 || d_k <= 0 || d_v <= 0)
    return fail(LA_ERR_INVALID_ARG, "la_decode_step: bad sizes B=%d H=%d d_k=%d d_v=%d", B, H,
                d_k, d_v);
  if (!decode_supported(d_k, d_v))
    return fail(LA_ERR_UNSUPPORTED,
                "la_decode_step: d_k=%d d_v=%d unsupported (need d_k = d_v in {16,32,64,128})",
                d_k, d_v);
  if ((size_t)B * H == 0) return ok();
  if (!q || !k || !v || !S || !o)
    return fail(LA_ERR_INVALID_ARG, "la_decode_step: q, k, v, S and o must be non-null");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(S) || !aligned16(o))
    return fail(LA_ERR_INVALID_ARG, "la_decode_step: tensors must start on a 16-byte boundary");
  DecodeArgs a{q, k, v, dtype, B, H, d_k, d_v, g_phi.load(), log_alpha, S, o,
               static_cast<cudaStream_t>(cuda_stream)};
  cudaError_t e = launch_decode(a);
  if (e != cudaSuccess) return cuda_fail(e, "la_decode_step");
  return ok();
}

size_t la_normalised_fwd_workspace_bytes(int B, int H, int L, int d_k, int d_v, int chunk,
                                         int dtype) {
  if (B <= 0 || H <= 0 || L <= 0 || !supported_d(d_k) || !supported_d(d_v)) return 0;
  PrefillArgs probe{};
  probe.dtype = dtype;
  probe.B = B;
  probe.H = H;
  probe.L = L;
  probe.dk = d_k;
  probe.dv = d_v;
  probe.chunk = chunk;
  if (prefill_tc_norm_supported(probe)) return prefill_tc_norm_workspace_bytes(B, H, L);
  return align256(la_chunk_fwd_workspace_bytes(B, H, L, d_k, d_v, chunk, dtype)) +
         normaliser_workspace_bytes(B, H, L, d_k);
}

la_status la_normalised_fwd(const void *q, const void *k, const void *v, int dtype, int B,
                            int H, int L, int d_k, int d_v, int chunk, int decay_kind,
                            const float *decay, const float *S0, const float *z0, void *O,
                            float *S_final, float *z_final, void *workspace, size_t ws_bytes,
                            void *cuda_stream) {
  const char *fn = "la_normalised_fwd";
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (decay_kind < LA_DECAY_NONE || decay_kind > LA_DECAY_GATE_LOGIT)
    return fail(LA_ERR_INVALID_ARG, "%s: unknown decay kind %d", fn, decay_kind);
  if (decay_kind != LA_DECAY_NONE && !decay)
    return fail(LA_ERR_INVALID_ARG, "%s: decay kind %d needs a decay pointer", fn, decay_kind);
  bool done = false;
  la_status s = check_variant(fn, q, k, v, dtype, B, H, L, d_k, d_v, chunk, true, S0, z0, O,
                              S_final, z_final, st, &done);
  if (s != LA_OK || done) return s;
  const int phi = g_phi.load();
  const float *dec = decay_kind == LA_DECAY_NONE ? nullptr : decay;
  {
    // One pass on the d = 64 tensor-core kernels: the denominator and z ride
    // with the numerator and the state as one more value column.
    PrefillArgs a{q, k, v, dtype, B, H, L, d_k, d_v, chunk, phi, decay_kind, dec, S0, O,
                  S_final, workspace, ws_bytes, st};
    if (prefill_tc_norm_supported(a)) {
      const size_t need = prefill_tc_norm_workspace_bytes(B, H, L);
      if (need > 0 && (!workspace || ws_bytes < need))
        return fail(LA_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                    workspace ? ws_bytes : (size_t)0);
      if (need > 0 && !aligned16(workspace))
        return fail(LA_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", fn);
      const char *why = nullptr;
      const cudaError_t e = launch_prefill_tc_norm(a, z0, z_final, &why);
      if (e != cudaSuccess) return cuda_fail(e, why ? why : fn);
      return ok();
    }
  }
  const size_t num_ws = la_chunk_fwd_workspace_bytes(B, H, L, d_k, d_v, chunk, dtype);
  const size_t need = align256(num_ws) + normaliser_workspace_bytes(B, H, L, d_k);
  if (!workspace || ws_bytes < need)
    return fail(LA_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                workspace ? ws_bytes : (size_t)0);
  if (!aligned16(workspace))
    return fail(LA_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", fn);
  // The numerator phi(q_t)^T S_t goes to O (and S_final) through the prefill
  // kernels; the normaliser then forms z and divides O in place.
  PrefillArgs a{q, k, v, dtype, B, H, L, d_k, d_v, chunk, phi, decay_kind, dec, S0, O,
                S_final, num_ws ? workspace : nullptr, num_ws, st};
  cudaError_t e;
  const char *why = nullptr;
  if (prefill_tc_supported(a)) {
    e = launch_prefill_tc(a, &why);
  } else {
    e = launch_prefill_simt(a);
  }
  if (e != cudaSuccess) return cuda_fail(e, why ? why : fn);
  NormaliserArgs n{q, k, dtype, B, H, L, d_k, d_v, phi, decay_kind, dec, z0, O, z_final,
                   static_cast<char *>(workspace) + align256(num_ws), st};
  e = launch_normaliser(n);
  if (e != cudaSuccess) return cuda_fail(e, fn);
  return ok();
}

size_t la_channel_gate_fwd_workspace_bytes(int B, int H, int L, int d_k, int d_v, int chunk,
                                           int dtype) {
  if (dtype != LA_BF16 || chunk != 64 || d_k != d_v) return 0;
  return channel_gate_tc_workspace_bytes(B, H, L, d_k);
}

la_status la_channel_gate_fwd(const void *q, const void *k, const void *v, int dtype, int B,
                              int H, int L, int d_k, int d_v, int chunk, const float *log_alpha,
                              const float *S0, void *O, float *S_final, void *workspace,
                              size_t ws_bytes, void *cuda_stream) {
  const char *fn = "la_channel_gate_fwd";
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  bool done = false;
  la_status s = check_variant(fn, q, k, v, dtype, B, H, L, d_k, d_v, chunk, true, S0, nullptr,
                              O, S_final, nullptr, st, &done);
  if (s != LA_OK || done) return s;
  if (!log_alpha) return fail(LA_ERR_INVALID_ARG, "%s: log_alpha must be non-null", fn);
  if (!aligned16(log_alpha))
    return fail(LA_ERR_INVALID_ARG, "%s: log_alpha must start on a 16-byte boundary", fn);
  if (workspace) {
    const size_t need = la_channel_gate_fwd_workspace_bytes(B, H, L, d_k, d_v, chunk, dtype);
    if (ws_bytes < need)
      return fail(LA_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                  ws_bytes);
    if (!aligned16(workspace))
      return fail(LA_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", fn);
  }
  VariantArgs a{VARIANT_CHANNEL_GATE, q, k, v, dtype, B, H, L, d_k, d_v, chunk, g_phi.load(),
                log_alpha, nullptr, S0, O, S_final, st};
  a.workspace = workspace;
  a.ws_bytes = workspace ? ws_bytes : 0;
  return run_variant(fn, a);
}

la_status la_delta_fwd(const void *q, const void *k, const void *v, int dtype, int B, int H,
                       int L, int d_k, int d_v, const float *beta, const float *log_alpha,
                       const float *S0, void *O, float *S_final, void *cuda_stream) {
  const char *fn = "la_delta_fwd";
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  bool done = false;
  la_status s = check_variant(fn, q, k, v, dtype, B, H, L, d_k, d_v, 0, false, S0, nullptr, O,
                              S_final, nullptr, st, &done);
  if (s != LA_OK || done) return s;
  if (!beta) return fail(LA_ERR_INVALID_ARG, "%s: beta must be non-null", fn);
  VariantArgs a{VARIANT_DELTA, q, k, v, dtype, B, H, L, d_k, d_v, 0, g_phi.load(), log_alpha,
                beta, S0, O, S_final, st};
  return run_variant(fn, a);
}

la_status la_causal_conv_fwd(const void *x, long long x_stride, int dtype, int B, int L, int D,
                             int width, const float *weight, const float *bias, int activation,
                             const int *lengths, const void *state0, void *y,
                             long long y_stride, void *state_final, void *cuda_stream) {
  const char *fn = "la_causal_conv_fwd";
  if (dtype != LA_F32 && dtype != LA_BF16)
    return fail(LA_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, dtype);
  if (B < 0 || L < 0 || D < 0)
    return fail(LA_ERR_INVALID_ARG, "%s: bad sizes B=%d L=%d D=%d", fn, B, L, D);
  if (activation != LA_ACT_NONE && activation != LA_ACT_SILU)
    return fail(LA_ERR_INVALID_ARG, "%s: activation %d is not none or silu", fn, activation);
  if (width < 2 || width > 8)
    return fail(LA_ERR_UNSUPPORTED, "%s: width %d outside 2..8", fn, width);
  if (L > kMaxLen || D > kMaxLen)
    return fail(LA_ERR_UNSUPPORTED, "%s: L=%d or D=%d above 2^30", fn, L, D);
  if (x_stride < D || y_stride < D)
    return fail(LA_ERR_INVALID_ARG, "%s: row strides %lld, %lld shorter than a row of %d", fn,
                x_stride, y_stride, D);
  if ((size_t)B * D == 0) return ok();
  const size_t elt = dtype == LA_F32 ? 4 : 2;
  if (!weight || (L > 0 && (!x || !y)))
    return fail(LA_ERR_INVALID_ARG, "%s: x, weight and y must be non-null", fn);
  if (!aligned_elt(x, elt) || !aligned_elt(y, elt) || !aligned_elt(state0, elt) ||
      !aligned_elt(state_final, elt) || !aligned_elt(lengths, 4))
    return fail(LA_ERR_INVALID_ARG, "%s: pointers must be aligned to their elements", fn);
  if (!aligned16(weight) || !aligned16(bias))
    return fail(LA_ERR_INVALID_ARG, "%s: weight and bias must be 16-byte aligned", fn);
  const long long rows = (long long)B * L;
  const size_t state_bytes = (size_t)B * (width - 1) * D * elt;
  const Rows xr{x, rows, D, x_stride, elt}, yr{y, rows, D, y_stride, elt};
  const Rows s0 = dense(state0, state_bytes), s1 = dense(state_final, state_bytes);
  const Rows par[] = {params(weight, (long long)D * width), params(bias, D), params(lengths, B)};
  if (overlap(yr, xr) || overlap(yr, s0) || overlap(yr, s1) || overlap(s1, xr) ||
      (state_final != state0 && overlap(s1, s0)) || overlap_any(yr, par) || overlap_any(s1, par))
    return fail(LA_ERR_INVALID_ARG, "%s: an output overlaps an input or another output", fn);
  ConvArgs a{x, x_stride, dtype, B, L, D, width, weight, bias, activation, lengths, state0, y,
             y_stride, state_final, static_cast<cudaStream_t>(cuda_stream)};
  cudaError_t e = launch_causal_conv(a);
  if (e != cudaSuccess) return cuda_fail(e, fn);
  return ok();
}

size_t la_selective_scan_fwd_workspace_bytes(int B, int L, int D, int N, int groups) {
  if (B <= 0 || L <= 0 || D <= 0 || N < 1 || N > 256 || groups < 1 || D % groups ||
      L > kMaxLen || D > kMaxLen)
    return 0;
  return selective_scan_workspace_bytes(B, L, D, N, groups);
}

la_status la_selective_scan_fwd(const void *x, long long x_stride, const void *dt,
                                long long dt_stride, const void *z, long long z_stride,
                                const void *Bm, long long b_stride, const void *Cm,
                                long long c_stride, int dtype, int B, int L, int D, int N,
                                int groups, const float *A, const float *dt_bias,
                                int dt_softplus, const float *skip, const float *h0,
                                const int *lengths, void *y, long long y_stride,
                                float *h_final, void *workspace, size_t ws_bytes,
                                void *cuda_stream) {
  const char *fn = "la_selective_scan_fwd";
  if (dtype != LA_F32 && dtype != LA_BF16)
    return fail(LA_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, dtype);
  if (B < 0 || L < 0 || D < 0 || N <= 0 || groups <= 0)
    return fail(LA_ERR_INVALID_ARG, "%s: bad sizes B=%d L=%d D=%d N=%d groups=%d", fn, B, L, D,
                N, groups);
  if (N > 256) return fail(LA_ERR_UNSUPPORTED, "%s: N=%d outside 1..256", fn, N);
  if (L > kMaxLen || D > kMaxLen)
    return fail(LA_ERR_UNSUPPORTED, "%s: L=%d or D=%d above 2^30", fn, L, D);
  if (D % groups)
    return fail(LA_ERR_UNSUPPORTED, "%s: D=%d is not a multiple of groups=%d", fn, D, groups);
  const long long gn = (long long)groups * N;
  if (x_stride < D || dt_stride < D || (z && z_stride < D) || y_stride < D || b_stride < gn ||
      c_stride < gn)
    return fail(LA_ERR_INVALID_ARG, "%s: a token stride is shorter than its row", fn);
  if ((size_t)B * D == 0) return ok();
  if (!aligned16(A) || !aligned16(dt_bias) || !aligned16(skip) || !aligned16(h0) ||
      !aligned16(h_final))
    return fail(LA_ERR_INVALID_ARG,
                "%s: A, dt_bias, skip and the states must be 16-byte aligned", fn);
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const size_t state_bytes = (size_t)B * D * N * sizeof(float);
  const Rows s0 = dense(h0, state_bytes), s1 = dense(h_final, state_bytes);
  if (h_final != h0 && overlap(s1, s0))
    return fail(LA_ERR_INVALID_ARG, "%s: h_final overlaps h0", fn);
  const Rows par[] = {params(A, (long long)D * N), params(dt_bias, D), params(skip, D),
                      params(lengths, B)};
  if (overlap_any(s1, par))
    return fail(LA_ERR_INVALID_ARG, "%s: h_final overlaps a parameter or lengths", fn);
  if (L == 0) {
    cudaError_t e = pass_through_state(h_final, h0, state_bytes, st);
    if (e != cudaSuccess) return cuda_fail(e, fn);
    return ok();
  }
  if (!x || !dt || !Bm || !Cm || !A || !y)
    return fail(LA_ERR_INVALID_ARG, "%s: x, dt, Bm, Cm, A and y must be non-null", fn);
  const size_t elt = dtype == LA_F32 ? 4 : 2;
  for (const void *p : {x, dt, z, Bm, Cm, static_cast<const void *>(y)})
    if (!aligned_elt(p, elt))
      return fail(LA_ERR_INVALID_ARG, "%s: pointers must be aligned to their elements", fn);
  if (!aligned_elt(lengths, 4))
    return fail(LA_ERR_INVALID_ARG, "%s: lengths must be 4-byte aligned", fn);
  const long long rows = (long long)B * L;
  const Rows yr{y, rows, D, y_stride, elt};
  const Rows in[] = {{x, rows, D, x_stride, elt},   {dt, rows, D, dt_stride, elt},
                     {z, rows, D, z_stride, elt},   {Bm, rows, gn, b_stride, elt},
                     {Cm, rows, gn, c_stride, elt}};
  if (overlap_any(yr, in) || overlap(yr, s0) || overlap_any(s1, in))
    return fail(LA_ERR_INVALID_ARG, "%s: an output overlaps an input", fn);
  if (overlap_any(yr, par))
    return fail(LA_ERR_INVALID_ARG, "%s: y overlaps a parameter or lengths", fn);
  if (overlap(yr, s1)) return fail(LA_ERR_INVALID_ARG, "%s: y overlaps h_final", fn);
  const size_t need = selective_scan_workspace_bytes(B, L, D, N, groups);
  if (workspace && ws_bytes < need)
    return fail(LA_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                ws_bytes);
  if (workspace && !aligned16(workspace))
    return fail(LA_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", fn);
  const Rows ws = dense(workspace, need);
  if (overlap(ws, yr) || overlap(ws, s0) || overlap(ws, s1) || overlap_any(ws, in) || overlap_any(ws, par))
    return fail(LA_ERR_INVALID_ARG, "%s: the workspace overlaps an input or an output", fn);
  ScanArgs a{x, dt, z, Bm, Cm, x_stride, dt_stride, z_stride, b_stride, c_stride, dtype, B, L,
             D, N, groups, A, dt_bias, dt_softplus, skip, h0, lengths, y, y_stride, h_final,
             need ? workspace : nullptr, st};
  cudaError_t e = launch_selective_scan(a);
  if (e != cudaSuccess) return cuda_fail(e, fn);
  return ok();
}

la_status la_gated_norm_fwd(const void *x, long long x_b_stride, long long x_h_stride,
                            long long x_t_stride, const void *gate, long long gate_stride,
                            int dtype, int B, int H, int L, int d, int norm, int activation,
                            int gate_first, const float *weight, const float *bias,
                            int weight_heads, float eps, void *y, long long y_stride,
                            void *cuda_stream) {
  const char *fn = "la_gated_norm_fwd";
  if (dtype != LA_F32 && dtype != LA_BF16)
    return fail(LA_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, dtype);
  if (B < 0 || H < 0 || L < 0 || d <= 0)
    return fail(LA_ERR_INVALID_ARG, "%s: bad sizes B=%d H=%d L=%d d=%d", fn, B, H, L, d);
  if (norm != LA_NORM_RMS && norm != LA_NORM_LAYER)
    return fail(LA_ERR_INVALID_ARG, "%s: unknown norm %d", fn, norm);
  if (activation < LA_ACT_NONE || activation > LA_ACT_SIGMOID)
    return fail(LA_ERR_INVALID_ARG, "%s: unknown activation %d", fn, activation);
  if (!(eps >= 0.f)) return fail(LA_ERR_INVALID_ARG, "%s: eps must be >= 0", fn);
  if (d > 16384) return fail(LA_ERR_UNSUPPORTED, "%s: d=%d outside 1..16384", fn, d);
  if (weight_heads != 1 && weight_heads != H)
    return fail(LA_ERR_INVALID_ARG, "%s: weight_heads=%d is neither 1 nor H=%d", fn,
                weight_heads, H);
  const long long width = (long long)H * d;
  if (x_b_stride < 0 || x_h_stride < 0 || x_t_stride < 0 || y_stride < width ||
      (gate && gate_stride < width))
    return fail(LA_ERR_INVALID_ARG, "%s: negative stride, or a row stride shorter than H*d", fn);
  if ((size_t)B * H == 0 || L == 0) return ok();
  if (!x || !y) return fail(LA_ERR_INVALID_ARG, "%s: x and y must be non-null", fn);
  const size_t elt = dtype == LA_F32 ? 4 : 2;
  if (!aligned_elt(x, elt) || !aligned_elt(gate, elt) || !aligned_elt(y, elt))
    return fail(LA_ERR_INVALID_ARG, "%s: pointers must be aligned to their elements", fn);
  if (!aligned16(weight) || !aligned16(bias))
    return fail(LA_ERR_INVALID_ARG, "%s: weight and bias must be 16-byte aligned", fn);
  const Heads yh = token_rows(y, B, H, L, d, y_stride, elt);
  const Rows par[] = {params(weight, (long long)weight_heads * d),
                      params(bias, (long long)weight_heads * d)};
  if (overlap(yh, heads_of(x, B, H, L, d, x_b_stride, x_h_stride, x_t_stride, elt)) ||
      (!(y == gate && y_stride == gate_stride) &&
       overlap(yh, token_rows(gate, B, H, L, d, gate_stride, elt))))
    return fail(LA_ERR_INVALID_ARG, "%s: y overlaps an input", fn);
  if (overlap_any(span_of(yh), par))
    return fail(LA_ERR_INVALID_ARG, "%s: y overlaps weight or bias", fn);
  GatedNormArgs a{x, x_b_stride, x_h_stride, x_t_stride, gate, gate_stride, dtype, B, H, L, d,
                  norm, activation, gate_first, weight, bias, weight_heads, eps, y, y_stride,
                  static_cast<cudaStream_t>(cuda_stream)};
  cudaError_t e = launch_gated_norm(a);
  if (e != cudaSuccess) return cuda_fail(e, fn);
  return ok();
}

la_status la_residual_norm_fwd(const void *x, int dtype, const void *residual, int res_dtype,
                               long long rows, int D, const float *post_weight,
                               const float *scale, float alpha, const float *weight,
                               const float *bias, int norm, float eps, void *y,
                               void *residual_out, void *cuda_stream) {
  const char *fn = "la_residual_norm_fwd";
  if (dtype != LA_F32 && dtype != LA_BF16)
    return fail(LA_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, dtype);
  if (res_dtype != LA_F32 && res_dtype != dtype)
    return fail(LA_ERR_INVALID_ARG, "%s: the residual's dtype %d is neither fp32 nor x's", fn,
                res_dtype);
  if (rows < 0 || D <= 0)
    return fail(LA_ERR_INVALID_ARG, "%s: bad sizes rows=%lld D=%d", fn, rows, D);
  if (norm != LA_NORM_RMS && norm != LA_NORM_LAYER)
    return fail(LA_ERR_INVALID_ARG, "%s: unknown norm %d", fn, norm);
  if (!(eps >= 0.f)) return fail(LA_ERR_INVALID_ARG, "%s: eps must be >= 0", fn);
  if (D > 16384) return fail(LA_ERR_UNSUPPORTED, "%s: D=%d outside 1..16384", fn, D);
  if (rows == 0) return ok();
  if (!x || !y) return fail(LA_ERR_INVALID_ARG, "%s: x and y must be non-null", fn);
  const size_t elt = dtype == LA_F32 ? 4 : 2, relt = res_dtype == LA_F32 ? 4 : 2;
  if (!aligned_elt(x, elt) || !aligned_elt(y, elt) || !aligned_elt(residual, relt) ||
      !aligned_elt(residual_out, relt))
    return fail(LA_ERR_INVALID_ARG, "%s: pointers must be aligned to their elements", fn);
  if (!aligned16(post_weight) || !aligned16(scale) || !aligned16(weight) || !aligned16(bias))
    return fail(LA_ERR_INVALID_ARG, "%s: parameters must be 16-byte aligned", fn);
  const Rows xr = dense(x, rows * D * elt), yr = dense(y, rows * D * elt);
  const Rows rr = dense(residual, rows * D * relt), ro = dense(residual_out, rows * D * relt);
  const Rows par[] = {params(post_weight, D), params(scale, D), params(weight, D),
                      params(bias, D)};
  if ((y != x && overlap(yr, xr)) || overlap(yr, rr) || overlap(yr, ro) || overlap(ro, xr) ||
      (residual_out != residual && overlap(ro, rr)) || overlap_any(yr, par) ||
      overlap_any(ro, par))
    return fail(LA_ERR_INVALID_ARG, "%s: an output overlaps an input or the other output", fn);
  ResidualNormArgs a{x, dtype, residual, res_dtype, rows, D, post_weight, scale, alpha, weight,
                     bias, norm, eps, y, residual_out, static_cast<cudaStream_t>(cuda_stream)};
  cudaError_t e = launch_residual_norm(a);
  if (e != cudaSuccess) return cuda_fail(e, fn);
  return ok();
}

la_status la_rotary_fwd(const void *q, long long q_b_stride, long long q_h_stride,
                        long long q_t_stride, int heads_q, const void *k, long long k_b_stride,
                        long long k_h_stride, long long k_t_stride, int heads_k, int dtype, int B,
                        int L, int d, int rotary_dim, int interleaved, const float *inv_freq,
                        float scale, const int *positions, const int *offsets,
                        const int *lengths, void *q_out, long long qo_b_stride,
                        long long qo_h_stride, long long qo_t_stride, void *k_out,
                        long long ko_b_stride, long long ko_h_stride, long long ko_t_stride,
                        void *cuda_stream) {
  return rotary("la_rotary_fwd",
                {{const_cast<void *>(q), q_b_stride, q_h_stride, q_t_stride},
                 {q_out, qo_b_stride, qo_h_stride, qo_t_stride},
                 {const_cast<void *>(k), k_b_stride, k_h_stride, k_t_stride},
                 {k_out, ko_b_stride, ko_h_stride, ko_t_stride},
                 heads_q, heads_k, dtype, B, L, d, rotary_dim, interleaved, 0, inv_freq, scale,
                 positions, offsets, lengths, static_cast<cudaStream_t>(cuda_stream)});
}

la_status la_rotary_bwd(const void *dq, long long q_b_stride, long long q_h_stride,
                        long long q_t_stride, int heads_q, const void *dk, long long k_b_stride,
                        long long k_h_stride, long long k_t_stride, int heads_k, int dtype, int B,
                        int L, int d, int rotary_dim, int interleaved, const float *inv_freq,
                        float scale, const int *positions, const int *offsets,
                        const int *lengths, void *dq_out, long long qo_b_stride,
                        long long qo_h_stride, long long qo_t_stride, void *dk_out,
                        long long ko_b_stride, long long ko_h_stride, long long ko_t_stride,
                        void *cuda_stream) {
  return rotary("la_rotary_bwd",
                {{const_cast<void *>(dq), q_b_stride, q_h_stride, q_t_stride},
                 {dq_out, qo_b_stride, qo_h_stride, qo_t_stride},
                 {const_cast<void *>(dk), k_b_stride, k_h_stride, k_t_stride},
                 {dk_out, ko_b_stride, ko_h_stride, ko_t_stride},
                 heads_q, heads_k, dtype, B, L, d, rotary_dim, interleaved, 1, inv_freq, scale,
                 positions, offsets, lengths, static_cast<cudaStream_t>(cuda_stream)});
}

la_status la_rotary_frequencies(int rotary_dim, double base, int scaling, double factor,
                                double trained_length, double fast, double slow, float *inv_freq,
                                float *scale) {
  const char *fn = "la_rotary_frequencies";
  if (rotary_dim < 2 || rotary_dim % 2)
    return fail(LA_ERR_INVALID_ARG, "%s: rotary_dim=%d is no positive even number", fn,
                rotary_dim);
  if (scaling < LA_ROTARY_PLAIN || scaling > LA_ROTARY_YARN)
    return fail(LA_ERR_INVALID_ARG, "%s: unknown scaling %d", fn, scaling);
  if (!inv_freq) return fail(LA_ERR_INVALID_ARG, "%s: inv_freq must be non-null", fn);
  if (!(base > 0) || !std::isfinite(base))
    return fail(LA_ERR_INVALID_ARG, "%s: base must be positive and finite", fn);
  if (scaling != LA_ROTARY_PLAIN && (!(factor >= 1) || !std::isfinite(factor)))
    return fail(LA_ERR_INVALID_ARG, "%s: factor must be finite and at least 1", fn);
  if (scaling == LA_ROTARY_YARN &&
      (!(trained_length > 0) || !(slow >= 0) || !(fast > slow) || !std::isfinite(fast) ||
       !std::isfinite(trained_length) || !(base > 1)))
    return fail(LA_ERR_INVALID_ARG,
                "%s: needs trained_length > 0, fast > slow >= 0 and base > 1", fn);
  if (scaling == LA_ROTARY_NTK && rotary_dim > 2)
    base *= std::pow(factor, rotary_dim / (rotary_dim - 2.0));
  // YaRN: the pairs (as real numbers) that make `fast` and `slow` turns, rounded away from one
  // another; both within the head's width, and never the same.
  double fast_pair = 0, slow_pair = 1;
  if (scaling == LA_ROTARY_YARN) {
    auto pair_of = [&](double turns) {
      return rotary_dim * std::log(trained_length / (turns * 6.283185307179586)) /
             (2 * std::log(base));
    };
    fast_pair = std::fmax(std::floor(pair_of(fast)), 0.0);
    slow_pair = std::fmin(std::ceil(pair_of(slow)), rotary_dim - 1.0);
    if (!(slow_pair > fast_pair)) slow_pair = fast_pair + 1e-3;
  }
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rotary_dim);
    if (scaling == LA_ROTARY_LINEAR) f /= factor;
    if (scaling == LA_ROTARY_YARN) {
      const double to_slow = std::fmin(std::fmax((i - fast_pair) / (slow_pair - fast_pair), 0.0), 1.0);
      f = f / factor * to_slow + f * (1 - to_slow);
    }
    inv_freq[i] = (float)f;
  }
  if (scale) *scale = scaling == LA_ROTARY_YARN ? (float)(1 + 0.1 * std::log(factor)) : 1.f;
  return ok();
}

size_t la_chunk_bwd_workspace_bytes(int B, int H, int L, int d_k, int d_v, int chunk, int dtype) {
  if (!chunk_bwd_sizes(B, H, L, d_k, d_v, chunk, dtype)) return 0;
  ChunkBwdArgs a{};
  a.dtype = dtype; a.B = B; a.H = H; a.L = L; a.dk = d_k; a.dv = d_v;
  return chunk_bwd_workspace_bytes(a);
}

size_t la_chunk_bwd_workspace_bytes_for(int B, int H, int L, int d_k, int d_v, int chunk, int dtype,
                                        int decay_kind, int ddecay, int dS0) {
  if (!chunk_bwd_sizes(B, H, L, d_k, d_v, chunk, dtype) || decay_kind < LA_DECAY_NONE ||
      decay_kind > LA_DECAY_GATE_LOGIT || (decay_kind == LA_DECAY_NONE && ddecay))
    return 0;
  ChunkBwdArgs a{};
  a.dtype = dtype; a.B = B; a.H = H; a.L = L; a.dk = d_k; a.dv = d_v;
  a.phi = g_phi.load(), a.decay_kind = decay_kind;
  return chunk_bwd_workspace_need(a, ddecay != 0, dS0 != 0);
}

la_status la_chunk_bwd(const void *q, const void *k, const void *v, int dtype, int B, int H,
                       int L, int d_k, int d_v, int chunk, int decay_kind, const float *decay,
                       const float *S0, const void *dO, const float *dS_final, void *dq, void *dk,
                       void *dv, float *ddecay, float *dS0, void *workspace, size_t ws_bytes,
                       void *cuda_stream) {
  const char *fn = "la_chunk_bwd";
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (dtype != LA_F32 && dtype != LA_BF16)
    return fail(LA_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, dtype);
  if (B < 0 || H < 0 || L < 0 || d_k <= 0 || d_v <= 0 || chunk <= 0)
    return fail(LA_ERR_INVALID_ARG, "%s: bad sizes B=%d H=%d L=%d d_k=%d d_v=%d chunk=%d", fn, B,
                H, L, d_k, d_v, chunk);
  if (decay_kind < LA_DECAY_NONE || decay_kind > LA_DECAY_GATE_LOGIT)
    return fail(LA_ERR_INVALID_ARG, "%s: unknown decay kind %d", fn, decay_kind);
  if (decay_kind == LA_DECAY_NONE && ddecay)
    return fail(LA_ERR_INVALID_ARG, "%s: ddecay without a decay", fn);
  if (!supported_d(d_k) || !supported_d(d_v))
    return fail(LA_ERR_UNSUPPORTED, "%s: d_k=%d d_v=%d not in {16,32,64,128}", fn, d_k, d_v);
  if (chunk > 64) return fail(LA_ERR_UNSUPPORTED, "%s: chunk %d > 64 is not supported", fn, chunk);
  if (L > kMaxLen || (long long)B * H > 0x7fffffffll)
    return fail(LA_ERR_UNSUPPORTED, "%s: L=%d above 2^30, or B*H above 2^31 - 1", fn, L);
  const size_t seqs = (size_t)B * H, states = seqs * d_k * d_v * sizeof(float);
  const size_t decays = decay_kind == LA_DECAY_NONE ? 0 : decay_kind == LA_DECAY_HEAD
                                                             ? (size_t)H : seqs * L;
  if (!aligned16(S0) || !aligned16(dS_final) || !aligned16(dS0) ||
      !aligned_elt(decay, 4) || !aligned_elt(ddecay, 4))
    return fail(LA_ERR_INVALID_ARG,
                "%s: states must be 16-byte aligned, decays to their elements", fn);
  const Rows s0 = dense(S0, states), sf = dense(dS_final, states), ds = dense(dS0, states);
  if (overlap(ds, s0) || overlap(ds, sf))
    return fail(LA_ERR_INVALID_ARG, "%s: dS0 overlaps S0 or dS_final", fn);
  if (seqs == 0 || L == 0) {  // no tokens: the state's gradient passes through
    cudaError_t e = seqs ? pass_through_state(dS0, dS_final, states, st) : cudaSuccess;
    if (e == cudaSuccess && ddecay && decay_kind == LA_DECAY_HEAD && H > 0)
      e = cudaMemsetAsync(ddecay, 0, (size_t)H * sizeof(float), st);
    if (e != cudaSuccess) return cuda_fail(e, fn);
    return ok();
  }
  if (!q || !k || !v || !dO || !dq || !dk || !dv)
    return fail(LA_ERR_INVALID_ARG, "%s: q, k, v, dO, dq, dk and dv must be non-null", fn);
  if (decay_kind != LA_DECAY_NONE && !decay)
    return fail(LA_ERR_INVALID_ARG, "%s: decay kind %d needs a decay pointer", fn, decay_kind);
  for (const void *p : {q, k, v, dO, static_cast<const void *>(dq),
                        static_cast<const void *>(dk), static_cast<const void *>(dv)})
    if (!aligned16(p))
      return fail(LA_ERR_INVALID_ARG, "%s: tensors must start on a 16-byte boundary", fn);
  const size_t elt = dtype == LA_F32 ? 4 : 2;
  const size_t nk = seqs * L * d_k * elt, nv = seqs * L * d_v * elt;
  const Rows in[] = {dense(q, nk), dense(k, nk), dense(v, nv), dense(dO, nv), s0,
                     dense(decay_kind == LA_DECAY_NONE ? nullptr : decay, decays * 4)};
  const Rows out[] = {dense(dq, nk), dense(dk, nk), dense(dv, nv), dense(ddecay, decays * 4), ds};
  for (int i = 0; i < 5; ++i) {
    bool bad = overlap_any(out[i], in) || overlap(out[i], sf);
    for (int j = 0; j < i; ++j) bad = bad || overlap(out[i], out[j]);
    if (bad)
      return fail(LA_ERR_INVALID_ARG, "%s: an output overlaps an input or another output", fn);
  }
  ChunkBwdArgs a{q, k, v, dO, dtype, B, H, L, d_k, d_v, g_phi.load(), decay_kind,
                 decay_kind == LA_DECAY_NONE ? nullptr : decay, S0, dS_final, dq, dk, dv, ddecay,
                 dS0, workspace, st};
  const size_t need = chunk_bwd_workspace_need(a, ddecay != nullptr, dS0 != nullptr);
  if (!workspace || ws_bytes < need)
    return fail(LA_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                workspace ? ws_bytes : (size_t)0);
  if (!aligned16(workspace))
    return fail(LA_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", fn);
  const Rows ws = dense(workspace, need);
  if (overlap_any(ws, in) || overlap_any(ws, out) || overlap(ws, sf))
    return fail(LA_ERR_INVALID_ARG, "%s: the workspace overlaps an input or an output", fn);
  cudaError_t e = launch_chunk_bwd(a);
  if (e != cudaSuccess) return cuda_fail(e, fn);
  return ok();
}

size_t la_gated_norm_bwd_workspace_bytes(int B, int H, int L, int d, int weight_heads) {
  if (B <= 0 || H <= 0 || L <= 0 || d < 1 || d > 16384 ||
      (weight_heads != 1 && weight_heads != H))
    return 0;
  return gated_norm_bwd_workspace_bytes(B, H, L, d, weight_heads);
}

la_status la_gated_norm_bwd(const void *dy, long long dy_stride, const void *x,
                            long long x_b_stride, long long x_h_stride, long long x_t_stride,
                            const void *gate, long long gate_stride, int dtype, int B, int H,
                            int L, int d, int norm, int activation, int gate_first,
                            const float *weight, const float *bias, int weight_heads, float eps,
                            void *dx, long long dx_b_stride, long long dx_h_stride,
                            long long dx_t_stride, void *dgate, long long dgate_stride,
                            float *dweight, float *dbias, void *workspace, size_t ws_bytes,
                            void *cuda_stream) {
  const char *fn = "la_gated_norm_bwd";
  if (dtype != LA_F32 && dtype != LA_BF16)
    return fail(LA_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, dtype);
  if (B < 0 || H < 0 || L < 0 || d <= 0)
    return fail(LA_ERR_INVALID_ARG, "%s: bad sizes B=%d H=%d L=%d d=%d", fn, B, H, L, d);
  if (norm != LA_NORM_RMS && norm != LA_NORM_LAYER)
    return fail(LA_ERR_INVALID_ARG, "%s: unknown norm %d", fn, norm);
  if (activation < LA_ACT_NONE || activation > LA_ACT_SIGMOID)
    return fail(LA_ERR_INVALID_ARG, "%s: unknown activation %d", fn, activation);
  if (!(eps >= 0.f)) return fail(LA_ERR_INVALID_ARG, "%s: eps must be >= 0", fn);
  if (d > 16384) return fail(LA_ERR_UNSUPPORTED, "%s: d=%d outside 1..16384", fn, d);
  if (H > 65535) return fail(LA_ERR_UNSUPPORTED, "%s: H=%d above 65535", fn, H);
  if (weight_heads != 1 && weight_heads != H)
    return fail(LA_ERR_INVALID_ARG, "%s: weight_heads=%d is neither 1 nor H=%d", fn,
                weight_heads, H);
  const long long width = (long long)H * d, wn = (long long)weight_heads * d;
  if (x_b_stride < 0 || x_h_stride < 0 || x_t_stride < 0 || dx_b_stride < 0 || dx_h_stride < 0 ||
      dx_t_stride < 0 || dy_stride < width || (gate && gate_stride < width) ||
      (dgate && dgate_stride < width))
    return fail(LA_ERR_INVALID_ARG, "%s: negative stride, or a row stride shorter than H*d", fn);
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (!aligned16(weight) || !aligned16(bias) || !aligned16(dweight) || !aligned16(dbias))
    return fail(LA_ERR_INVALID_ARG, "%s: parameters and their gradients must be 16-byte aligned",
                fn);
  if ((size_t)B * H == 0 || L == 0) {  // no rows: the sums over them are zero
    for (float *p : {dweight, dbias})
      if (p && wn > 0) {
        cudaError_t e = cudaMemsetAsync(p, 0, wn * sizeof(float), st);
        if (e != cudaSuccess) return cuda_fail(e, fn);
      }
    return ok();
  }
  if (!dy || !x || !dx) return fail(LA_ERR_INVALID_ARG, "%s: dy, x and dx must be non-null", fn);
  if (!gate != !dgate)
    return fail(LA_ERR_INVALID_ARG, "%s: dgate goes with gate: both or none", fn);
  const size_t elt = dtype == LA_F32 ? 4 : 2;
  for (const void *p : {dy, x, gate, static_cast<const void *>(dx),
                        static_cast<const void *>(dgate)})
    if (!aligned_elt(p, elt))
      return fail(LA_ERR_INVALID_ARG, "%s: pointers must be aligned to their elements", fn);
  if (!own_places(B, H, L, d, dx_b_stride, dx_h_stride, dx_t_stride))
    return fail(LA_ERR_INVALID_ARG, "%s: dx's strides put two elements in one place", fn);
  const Heads in[] = {token_rows(dy, B, H, L, d, dy_stride, elt),
                      heads_of(x, B, H, L, d, x_b_stride, x_h_stride, x_t_stride, elt),
                      token_rows(gate, B, H, L, d, gate_stride, elt)};
  const Heads dxh = heads_of(dx, B, H, L, d, dx_b_stride, dx_h_stride, dx_t_stride, elt);
  const Heads dzh = token_rows(dgate, B, H, L, d, dgate_stride, elt);
  const Rows par[] = {params(weight, wn), params(bias, wn)};
  const Rows span[] = {span_of(in[0]), span_of(in[1]), span_of(in[2]), span_of(dxh), span_of(dzh)};
  const Rows dw = params(dweight, wn), dbr = params(dbias, wn);
  const bool x_place = dx == x && (B == 1 || dx_b_stride == x_b_stride) &&
                       (H == 1 || dx_h_stride == x_h_stride) &&
                       (L == 1 || dx_t_stride == x_t_stride);
  const bool dy_place = dgate && dgate == dy && dgate_stride == dy_stride;
  const bool z_place = dgate && dgate == gate && dgate_stride == gate_stride;
  if (overlap(dxh, in[0]) || (!x_place && overlap(dxh, in[1])) || overlap(dxh, in[2]) ||
      (!dy_place && overlap(dzh, in[0])) || overlap(dzh, in[1]) ||
      (!z_place && overlap(dzh, in[2])) || overlap(dxh, dzh) || overlap_any(span[3], par) ||
      overlap_any(span[4], par))
    return fail(LA_ERR_INVALID_ARG, "%s: an output overlaps an input or another output", fn);
  for (const Rows &w : {dw, dbr})
    if (overlap_any(w, span) || overlap_any(w, par))
      return fail(LA_ERR_INVALID_ARG, "%s: an output overlaps an input or another output", fn);
  if (overlap(dw, dbr)) return fail(LA_ERR_INVALID_ARG, "%s: dweight and dbias overlap", fn);
  if (dweight || dbias) {
    const size_t need = gated_norm_bwd_workspace_bytes(B, H, L, d, weight_heads);
    if (!workspace || ws_bytes < need)
      return fail(LA_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                  workspace ? ws_bytes : (size_t)0);
    if (!aligned16(workspace))
      return fail(LA_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", fn);
    const Rows ws = dense(workspace, need);
    if (overlap_any(ws, span) || overlap_any(ws, par) || overlap(ws, dw) || overlap(ws, dbr))
      return fail(LA_ERR_INVALID_ARG, "%s: the workspace overlaps an input or an output", fn);
  }
  GatedNormBwdArgs a{dy, dy_stride, x, x_b_stride, x_h_stride, x_t_stride, gate, gate_stride,
                     dtype, B, H, L, d, norm, activation, gate_first, weight, bias, weight_heads,
                     eps, dx, dx_b_stride, dx_h_stride, dx_t_stride, dgate, dgate_stride,
                     dweight, dbias, workspace, st};
  cudaError_t e = launch_gated_norm_bwd(a);
  if (e != cudaSuccess) return cuda_fail(e, fn);
  return ok();
}

size_t la_residual_norm_bwd_workspace_bytes(long long rows, int D) {
  return rows <= 0 || D < 1 || D > 16384 ? 0 : residual_norm_bwd_workspace_bytes(rows, D);
}

la_status la_residual_norm_bwd(const void *dy, int dtype, const void *r, const void *dr,
                               int res_dtype, const void *x, long long rows, int D,
                               const float *post_weight, const float *scale, float alpha,
                               const float *weight, int norm, float eps, void *dx,
                               void *dresidual, float *dweight, float *dbias,
                               float *dpost_weight, float *dscale, void *workspace,
                               size_t ws_bytes, void *cuda_stream) {
  const char *fn = "la_residual_norm_bwd";
  if (dtype != LA_F32 && dtype != LA_BF16)
    return fail(LA_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, dtype);
  if (res_dtype != LA_F32 && res_dtype != dtype)
    return fail(LA_ERR_INVALID_ARG, "%s: the residual's dtype %d is neither fp32 nor dy's", fn,
                res_dtype);
  if (rows < 0 || D <= 0)
    return fail(LA_ERR_INVALID_ARG, "%s: bad sizes rows=%lld D=%d", fn, rows, D);
  if (norm != LA_NORM_RMS && norm != LA_NORM_LAYER)
    return fail(LA_ERR_INVALID_ARG, "%s: unknown norm %d", fn, norm);
  if (!(eps >= 0.f)) return fail(LA_ERR_INVALID_ARG, "%s: eps must be >= 0", fn);
  if (D > 16384) return fail(LA_ERR_UNSUPPORTED, "%s: D=%d outside 1..16384", fn, D);
  if ((!post_weight && dpost_weight) || (!scale && dscale))
    return fail(LA_ERR_INVALID_ARG, "%s: a gradient of a parameter that is not there", fn);
  float *const grads[] = {dweight, dbias, dpost_weight, dscale};
  for (const void *p : {static_cast<const void *>(post_weight), static_cast<const void *>(scale),
                        static_cast<const void *>(weight), static_cast<const void *>(dweight),
                        static_cast<const void *>(dbias),
                        static_cast<const void *>(dpost_weight),
                        static_cast<const void *>(dscale)})
    if (!aligned16(p))
      return fail(LA_ERR_INVALID_ARG,
                  "%s: parameters and their gradients must be 16-byte aligned", fn);
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (rows == 0) {  // the sums over no rows are zero
    for (float *p : grads)
      if (p) {
        cudaError_t e = cudaMemsetAsync(p, 0, (size_t)D * sizeof(float), st);
        if (e != cudaSuccess) return cuda_fail(e, fn);
      }
    return ok();
  }
  if (!dy || !r || !dx) return fail(LA_ERR_INVALID_ARG, "%s: dy, r and dx must be non-null", fn);
  if (!x && (post_weight || dscale))
    return fail(LA_ERR_INVALID_ARG, "%s: a post norm and dscale need x", fn);
  const size_t elt = dtype == LA_F32 ? 4 : 2, relt = res_dtype == LA_F32 ? 4 : 2;
  if (!aligned_elt(dy, elt) || !aligned_elt(x, elt) || !aligned_elt(dx, elt) ||
      !aligned_elt(r, relt) || !aligned_elt(dr, relt) || !aligned_elt(dresidual, relt))
    return fail(LA_ERR_INVALID_ARG, "%s: pointers must be aligned to their elements", fn);
  const size_t n = (size_t)rows * D;
  const Rows dyr = dense(dy, n * elt), xr = dense(x, n * elt), rr = dense(r, n * relt),
             drr = dense(dr, n * relt), dxr = dense(dx, n * elt), dres = dense(dresidual, n * relt);
  const Rows par[] = {params(post_weight, D), params(scale, D), params(weight, D)};
  if ((dx != dy && overlap(dxr, dyr)) || (dx != x && overlap(dxr, xr)) || overlap(dxr, rr) ||
      overlap(dxr, drr) || overlap(dres, dyr) || overlap(dres, xr) || overlap(dres, rr) ||
      (dresidual != dr && overlap(dres, drr)) || overlap(dxr, dres) || overlap_any(dxr, par) ||
      overlap_any(dres, par))
    return fail(LA_ERR_INVALID_ARG, "%s: an output overlaps an input or another output", fn);
  bool sums = false;
  for (int i = 0; i < 4; ++i) {
    const Rows g = params(grads[i], D);
    sums = sums || grads[i];
    bool bad = overlap_any(g, par);
    for (const Rows &o : {dyr, xr, rr, drr, dxr, dres}) bad = bad || overlap(g, o);
    for (int j = 0; j < i; ++j) bad = bad || overlap(g, params(grads[j], D));
    if (bad)
      return fail(LA_ERR_INVALID_ARG, "%s: an output overlaps an input or another output", fn);
  }
  if (sums) {
    const size_t need = residual_norm_bwd_workspace_bytes(rows, D);
    if (!workspace || ws_bytes < need)
      return fail(LA_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                  workspace ? ws_bytes : (size_t)0);
    if (!aligned16(workspace))
      return fail(LA_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", fn);
    const Rows ws = dense(workspace, need);
    bool bad = overlap_any(ws, par);
    for (const Rows &o : {dyr, xr, rr, drr, dxr, dres}) bad = bad || overlap(ws, o);
    for (float *g : grads) bad = bad || overlap(ws, params(g, D));
    if (bad)
      return fail(LA_ERR_INVALID_ARG, "%s: the workspace overlaps an input or an output", fn);
  }
  ResidualNormBwdArgs a{dy, dtype, r, dr, res_dtype, x, rows, D, post_weight, scale, alpha,
                        weight, norm, eps, dx, dresidual, dweight, dbias, dpost_weight, dscale,
                        workspace, st};
  cudaError_t e = launch_residual_norm_bwd(a);
  if (e != cudaSuccess) return cuda_fail(e, fn);
  return ok();
}

la_status la_device_status(void *cuda_stream) {
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(cuda_stream));
  if (e != cudaSuccess) return cuda_fail(e, "la_device_status: stream synchronize");
  unsigned int word = 0, zero = 0;
  e = cudaMemcpyFromSymbol(&word, g_device_error, sizeof word);
  if (e != cudaSuccess) return cuda_fail(e, "la_device_status: read error word");
  if (word == 0) return ok();
  e = cudaMemcpyToSymbol(g_device_error, &zero, sizeof zero);
  if (e != cudaSuccess) return cuda_fail(e, "la_device_status: clear error word");
  return fail(LA_ERR_DEVICE_TIMEOUT, "bounded wait timed out in %s (wait site %u)",
              kernel_name(word & 0xffu), (word >> 8) & 0xffu);
}

la_status la_selftest_wait_timeout(unsigned int spin_limit, void *cuda_stream) {
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e = launch_wait_timeout_selftest(spin_limit, st);
  if (e != cudaSuccess) return cuda_fail(e, "la_selftest_wait_timeout: launch");
  return la_device_status(cuda_stream);
}

const char *la_last_error(void) { return g_msg; }

}  // extern "C"
