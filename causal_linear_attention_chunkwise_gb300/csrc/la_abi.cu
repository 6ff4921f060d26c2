// la_abi.cu -- the extern "C" boundary: argument validation, dispatch to the
// kernel launchers, the process-wide feature map, error reporting.
#include <atomic>
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

const char *kernel_name(unsigned int id) {
  switch (id) {
    case KID_PREFILL_TC_STATE: return "prefill segment-state kernel";
    case KID_PREFILL_TC_OUT: return "prefill chunk-output kernel";
    case KID_SELFTEST: return "wait-timeout self-test kernel";
    case KID_NONCAUSAL: return "non-causal output kernel";
    case KID_CHANNEL_GATE_TC: return "per-channel gate tensor-core kernel";
    case KID_DELTA_TC: return "delta-rule tensor-core kernel";
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
  const long long rows = (long long)B * L;
  const Rows yr{y, rows, width, y_stride, elt}, gr{gate, rows, width, gate_stride, elt};
  const long long span = (B - 1) * x_b_stride + (H - 1) * x_h_stride + (L - 1) * x_t_stride + d;
  Rows xr{x, 1, span, span, elt};
  if ((H == 1 || x_h_stride == d) && (B == 1 || x_b_stride == L * x_t_stride) &&
      (L == 1 || x_t_stride >= width))
    xr = {x, rows, width, rows == 1 ? width : L == 1 ? x_b_stride : x_t_stride,
          elt};  // token-major rows, which may be a slice
  const Rows par[] = {params(weight, (long long)weight_heads * d),
                      params(bias, (long long)weight_heads * d)};
  if (overlap(yr, xr) || (!(y == gate && y_stride == gate_stride) && overlap(yr, gr)) ||
      overlap_any(yr, par))
    return fail(LA_ERR_INVALID_ARG, "%s: y overlaps an input", fn);
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
