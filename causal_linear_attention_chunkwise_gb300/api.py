"""Python binding of the C ABI, with the same names.  Argument marshalling only:
tensors become device pointers, torch supplies output memory and the current
CUDA stream, and every step of the computation runs in the library's kernels.

Host (CPU) tensors are accepted too: they are copied to the current device,
the same kernels run, and the outputs are copied back (this is the
end-to-end path the benchmark times with host buffers).
"""
from __future__ import annotations

import torch

from . import _native

PHI = {"identity": 0, "elu1": 1}
DTYPE = {torch.float32: 0, torch.bfloat16: 1}
DECAY = {"none": 0, "head": 1, "token": 2, "logit": 3}
ACT = {"none": 0, "silu": 1, "sigmoid": 2}
NORM = {"rms": 0, "layer": 1}
ROTARY = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3}

LA_OK, LA_ERR_INVALID_ARG, LA_ERR_UNSUPPORTED, LA_ERR_CUDA, LA_ERR_DEVICE_TIMEOUT = range(5)


class LAError(RuntimeError):
    """A non-zero la_status, with the library's message."""

    def __init__(self, status: int, message: str):
        super().__init__(f"la_status {status}: {message}")
        self.status = status


def _check(status: int):
    if status != LA_OK:
        raise LAError(status, _native.load().la_last_error().decode())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    if torch.cuda.is_initialized():
        return _current_stream(_current_device())
    return torch.cuda.current_stream().cuda_stream


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("expected CUDA tensors")
        if t is not None and not t.is_contiguous():
            raise ValueError("expected contiguous tensors")


def la_set_feature_map(phi) -> None:
    """Select phi ("identity" | "elu1" or 0 | 1) for all later calls."""
    _check(_native.load().la_set_feature_map(PHI.get(phi, phi)))


def la_get_feature_map() -> int:
    return _native.load().la_get_feature_map()


def la_chunk_fwd_workspace_bytes(B, H, L, d_k, d_v, chunk=64, dtype=torch.bfloat16) -> int:
    return int(_native.load().la_chunk_fwd_workspace_bytes(B, H, L, d_k, d_v, chunk,
                                                           DTYPE[dtype]))


def la_chunk_fwd_kernel_count(B, H, L, d_k, d_v, chunk=64, dtype=torch.bfloat16) -> int:
    return int(_native.load().la_chunk_fwd_kernel_count(B, H, L, d_k, d_v, chunk, DTYPE[dtype]))


def _new(shape, dtype, device, stream, zero=False):
    """A tensor on the stream that the call runs on."""
    make = torch.zeros if zero else torch.empty
    if stream is None or stream.cuda_stream == _current_stream(device.index):
        return make(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=device)


def _workspace(nbytes, device, stream=None):
    """Workspace of one call, from the allocator on the call's stream: calls of two
    threads on one stream, whose launches may interleave, get two buffers, a
    captured call one of its graph's own, and a freed one goes to no call before
    this one on the stream has run."""
    return _new((nbytes,), torch.uint8, device, stream) if nbytes else None


def la_chunk_fwd(q, k, v, chunk=64, decay_kind="none", decay=None, S0=None, O=None,
                 S_final=None, want_final_state=True, workspace=None, stream=None):
    """Chunkwise causal linear attention over [B,H,L,d] sequences.

    Returns ``(O, S_final)`` (``S_final`` is None when ``want_final_state`` is
    false and no buffer is given).  ``decay_kind``: "none" | "head" (decay =
    fp32 [H] log gamma) | "token" (fp32 [B,H,L] log alpha) | "logit" (fp32
    [B,H,L] gate logits g).  ``S0``: fp32 [B,H,d_k,d_v] or None.
    """
    if not q.is_cuda:
        return _chunk_fwd_host(q, k, v, chunk, decay_kind, decay, S0, want_final_state)
    B, H, L, dk = q.shape
    dv = v.shape[-1]
    if k.shape != q.shape or v.shape[:3] != q.shape[:3] or v.dtype != q.dtype or k.dtype != q.dtype:
        raise ValueError("q, k, v must agree in [B,H,L] and dtype")
    if O is None:
        O = torch.empty(B, H, L, dv, dtype=q.dtype, device=q.device)
    if S_final is None and want_final_state:
        S_final = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device)
    _need_cuda(q, k, v, decay, S0, O, S_final)
    lib = _native.load()
    ws_need = la_chunk_fwd_workspace_bytes(B, H, L, dk, dv, chunk, q.dtype)
    if workspace is None:
        workspace = _workspace(ws_need, q.device, stream)
    _check(lib.la_chunk_fwd(
        _ptr(q), _ptr(k), _ptr(v), DTYPE[q.dtype], B, H, L, dk, dv, chunk,
        DECAY[decay_kind], _ptr(decay), _ptr(S0), _ptr(O), _ptr(S_final),
        _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(),
        _stream(stream)))
    return O, S_final


def la_noncausal_fwd_workspace_bytes(B, H, L, d_k, d_v) -> int:
    return int(_native.load().la_noncausal_fwd_workspace_bytes(B, H, L, d_k, d_v))


def la_noncausal_fwd(q, k, v, O=None, S=None, want_state=True, workspace=None, stream=None):
    """Non-causal linear attention O = phi(Q) (phi(K)^T V) over [B,H,L,d] bf16
    sequences on the GPU.  Returns ``(O, S)`` with S = phi(K)^T V, fp32
    [B,H,d,d] (None when ``want_state`` is false and no buffer is given)."""
    B, H, L, dk = q.shape
    dv = v.shape[-1]
    if k.shape != q.shape or v.shape[:3] != q.shape[:3] or v.dtype != q.dtype or k.dtype != q.dtype:
        raise ValueError("q, k, v must agree in [B,H,L] and dtype")
    if O is None:
        O = torch.empty(B, H, L, dv, dtype=q.dtype, device=q.device)
    if S is None and want_state:
        S = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device)
    _need_cuda(q, k, v, O, S)
    lib = _native.load()
    if workspace is None:
        workspace = _workspace(la_noncausal_fwd_workspace_bytes(B, H, L, dk, dv), q.device,
                               stream)
    _check(lib.la_noncausal_fwd(
        _ptr(q), _ptr(k), _ptr(v), DTYPE[q.dtype], B, H, L, dk, dv, _ptr(O), _ptr(S),
        _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(),
        _stream(stream)))
    return O, S


def la_chunk_fwd_noalloc(q, k, v, chunk=64, decay_kind="none", decay=None, S0=None, O=None,
                         S_final=None, want_final_state=True, stream=None):
    """la_chunk_fwd without a caller workspace, for callers that cannot
    allocate device memory at call time: the library's fixed static scratch
    (la_chunk_fwd_noalloc_scratch_bytes() bytes per GPU) holds the segment
    states.  Calls on one device share that scratch, so calls that may run
    concurrently on the GPU must be ordered by the caller.  Output buffers
    are allocated here only when not given; pass O and S_final to allocate
    nothing at all."""
    B, H, L, dk = q.shape
    dv = v.shape[-1]
    if O is None:
        O = torch.empty(B, H, L, dv, dtype=q.dtype, device=q.device)
    if S_final is None and want_final_state:
        S_final = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device)
    _need_cuda(q, k, v, decay, S0, O, S_final)
    _check(_native.load().la_chunk_fwd_noalloc(
        _ptr(q), _ptr(k), _ptr(v), DTYPE[q.dtype], B, H, L, dk, dv, chunk, DECAY[decay_kind],
        _ptr(decay), _ptr(S0), _ptr(O), _ptr(S_final), _stream(stream)))
    return O, S_final


def la_chunk_fwd_noalloc_prepare():
    """Look up the static scratch on the current device (which is where lazy
    module loading reserves it).  Call once per device at start-up, before
    the point where the caller may no longer allocate."""
    _check(_native.load().la_chunk_fwd_noalloc_prepare())


def la_chunk_fwd_noalloc_scratch_bytes() -> int:
    return int(_native.load().la_chunk_fwd_noalloc_scratch_bytes())


def _chunk_fwd_host(q, k, v, chunk, decay_kind, decay, S0, want_final_state):
    dev = torch.device("cuda", torch.cuda.current_device())
    to = lambda t: None if t is None else t.to(dev, non_blocking=True)  # noqa: E731
    O, Sf = la_chunk_fwd(to(q), to(k), to(v), chunk, decay_kind, to(decay), to(S0),
                         want_final_state=want_final_state)
    O_h = torch.empty(O.shape, dtype=O.dtype, pin_memory=True)
    O_h.copy_(O, non_blocking=True)
    Sf_h = None
    if Sf is not None:
        Sf_h = torch.empty(Sf.shape, dtype=Sf.dtype, pin_memory=True)
        Sf_h.copy_(Sf, non_blocking=True)
    torch.cuda.current_stream().synchronize()
    return O_h, Sf_h


def la_decode_step(q, k, v, S, log_alpha=None, o=None, stream=None):
    """One decode step: S <- alpha S + phi(k) v^T in place, returns o = phi(q)^T S.
    q, k [B,H,d_k], v [B,H,d_v], S fp32 [B,H,d_k,d_v], log_alpha fp32 [B,H]."""
    B, H, dk = q.shape
    dv = v.shape[-1]
    if o is None:
        o = torch.empty(B, H, dv, dtype=q.dtype, device=q.device)
    _need_cuda(q, k, v, S, log_alpha, o)
    if S.dtype != torch.float32:
        raise ValueError("the state S must be fp32")
    _check(_native.load().la_decode_step(
        _ptr(q), _ptr(k), _ptr(v), DTYPE[q.dtype], B, H, dk, dv, _ptr(log_alpha), _ptr(S),
        _ptr(o), _stream(stream)))
    return o


def _state_bufs(q, v, want, S_final, extra=False, z_final=None):
    B, H, _, dk = q.shape
    dv = v.shape[-1]
    if S_final is None and want:
        S_final = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device)
    if extra and z_final is None and want:
        z_final = torch.empty(B, H, dk, dtype=torch.float32, device=q.device)
    return S_final, z_final


def _qkv(q, k, v, O):
    if k.shape != q.shape or v.shape[:3] != q.shape[:3] or v.dtype != q.dtype or k.dtype != q.dtype:
        raise ValueError("q, k, v must agree in [B,H,L] and dtype")
    B, H, L, _ = q.shape
    if O is None:
        O = torch.empty(B, H, L, v.shape[-1], dtype=q.dtype, device=q.device)
    return O


def la_normalised_fwd_workspace_bytes(B, H, L, d_k, d_v, chunk=64, dtype=torch.bfloat16) -> int:
    return int(_native.load().la_normalised_fwd_workspace_bytes(B, H, L, d_k, d_v, chunk,
                                                                DTYPE[dtype]))


def la_normalised_fwd(q, k, v, chunk=64, decay_kind="none", decay=None, S0=None, z0=None,
                      O=None, S_final=None, z_final=None, want_final_state=True,
                      workspace=None, stream=None):
    """Normalised form o_t = phi(q_t)^T S_t / phi(q_t)^T z_t over [B,H,L,d]
    sequences, z the decayed key sum.  Returns ``(O, S_final, z_final)``.
    ``S0`` fp32 [B,H,d_k,d_v], ``z0`` fp32 [B,H,d_k]; the outputs may be the
    same tensors as the inputs (with L = 1 that is one decode step)."""
    O = _qkv(q, k, v, O)
    S_final, z_final = _state_bufs(q, v, want_final_state, S_final, True, z_final)
    _need_cuda(q, k, v, decay, S0, z0, O, S_final, z_final)
    B, H, L, dk = q.shape
    dv = v.shape[-1]
    if workspace is None:
        workspace = _workspace(la_normalised_fwd_workspace_bytes(B, H, L, dk, dv, chunk, q.dtype),
                               q.device, stream)
    _check(_native.load().la_normalised_fwd(
        _ptr(q), _ptr(k), _ptr(v), DTYPE[q.dtype], B, H, L, dk, dv, chunk,
        DECAY[decay_kind], _ptr(decay), _ptr(S0), _ptr(z0), _ptr(O), _ptr(S_final),
        _ptr(z_final), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(),
        _stream(stream)))
    return O, S_final, z_final


def la_channel_gate_fwd_workspace_bytes(B, H, L, d_k, d_v, chunk=64, dtype=torch.bfloat16) -> int:
    return int(_native.load().la_channel_gate_fwd_workspace_bytes(B, H, L, d_k, d_v, chunk,
                                                                  DTYPE[dtype]))


def la_channel_gate_fwd(q, k, v, log_alpha, chunk=64, S0=None, O=None, S_final=None,
                        want_final_state=True, workspace=None, segments=True, stream=None):
    """Per-channel gate S_t = diag(alpha_t) S_{t-1} + phi(k_t) v_t^T with
    ``log_alpha`` fp32 [B,H,L,d_k].  Returns ``(O, S_final)``.  With
    ``segments`` (the default) a workspace lets the library run each
    sequence as several segments side by side; ``segments=False`` runs each
    sequence in one piece."""
    O = _qkv(q, k, v, O)
    S_final, _ = _state_bufs(q, v, want_final_state, S_final)
    _need_cuda(q, k, v, log_alpha, S0, O, S_final)
    B, H, L, dk = q.shape
    dv = v.shape[-1]
    if log_alpha.shape != (B, H, L, dk) or log_alpha.dtype != torch.float32:
        raise ValueError("log_alpha must be fp32 [B,H,L,d_k]")
    if workspace is None and segments:
        workspace = _workspace(la_channel_gate_fwd_workspace_bytes(B, H, L, dk, dv, chunk, q.dtype),
                               q.device, stream)
    _check(_native.load().la_channel_gate_fwd(
        _ptr(q), _ptr(k), _ptr(v), DTYPE[q.dtype], B, H, L, dk, dv, chunk,
        _ptr(log_alpha), _ptr(S0), _ptr(O), _ptr(S_final), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(),
        _stream(stream)))
    return O, S_final


def la_delta_fwd(q, k, v, beta, log_alpha=None, S0=None, O=None, S_final=None,
                 want_final_state=True, stream=None):
    """(Gated) delta rule S <- alpha (S - beta k (k^T S)) + beta k v^T,
    o = phi(q)^T S, token by token; ``beta`` and ``log_alpha`` fp32 [B,H,L]
    (``log_alpha`` None: alpha = 1).  Returns ``(O, S_final)``."""
    O = _qkv(q, k, v, O)
    S_final, _ = _state_bufs(q, v, want_final_state, S_final)
    _need_cuda(q, k, v, beta, log_alpha, S0, O, S_final)
    B, H, L, dk = q.shape
    for t in (beta, log_alpha):
        if t is not None and (t.shape != (B, H, L) or t.dtype != torch.float32):
            raise ValueError("beta and log_alpha must be fp32 [B,H,L]")
    _check(_native.load().la_delta_fwd(
        _ptr(q), _ptr(k), _ptr(v), DTYPE[q.dtype], B, H, L, dk, v.shape[-1], _ptr(beta),
        _ptr(log_alpha), _ptr(S0), _ptr(O), _ptr(S_final), _stream(stream)))
    return O, S_final


# ---------------------------------------------------------------- state space block
# These calls also serve single tokens, where the time of the checks counts:
# each tensor is asked for no more than it has to be.
def _device_of(x, *ts):
    """The current device (the one the library launches on), where every tensor
    given has to lie."""
    dev = x.get_device()
    if dev < 0:
        raise ValueError("expected CUDA tensors")
    for t in ts:
        if t is not None and t.get_device() != dev:
            raise ValueError("expected CUDA tensors on one device")
    if dev != _current_device():
        raise ValueError("expected tensors on the current device")
    return dev


# What torch.cuda.current_device and current_stream ask, without their objects (a
# CUDA tensor is at hand, so CUDA is initialised).
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda dev: torch.cuda.current_stream(dev).cuda_stream)


_INT_MAX = 2 ** 31 - 1  # sizes cross the C ABI as int, which ctypes would cut silently


def _too_large(*sizes):
    return ValueError(f"a size above 2^31 - 1 among {list(sizes)}")


def _param(t, shape, what):
    if t.dtype != torch.float32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous fp32 {list(shape)}")
    return t.data_ptr()


def _row_stride(t, shape, dtype, what):
    """Elements between the tokens of ``t`` = [B,L,...] (token rows contiguous,
    sequences L rows apart), after its shape and dtype have been checked."""
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype} {list(shape)}")
    if t.is_contiguous():
        return shape[2] if len(shape) == 3 else shape[2] * shape[3]
    st = t.stride()
    inner = 1
    for n, s in zip(reversed(shape[2:]), reversed(st[2:])):
        if n != 1 and s != inner:
            raise ValueError(f"the values of one token of {what} must be contiguous")
        inner *= n
    row = st[1] if shape[1] > 1 else st[0] if shape[0] > 1 else inner
    if row < inner or (shape[0] > 1 and st[0] != shape[1] * row):
        raise ValueError(f"the tokens of {what} must lie evenly apart")
    return row


def _lengths_ptr(lengths, B):
    if lengths.dtype != torch.int32 or lengths.shape != (B,) or not lengths.is_contiguous():
        raise ValueError("lengths must be contiguous int32 [B]")
    return lengths.data_ptr()


def _conv_state(t, shape, dtype):
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError("the states must be contiguous [B,W-1,D] in x's dtype")
    return t.data_ptr()


def la_causal_conv_fwd(x, weight, bias=None, activation="silu", state0=None, lengths=None,
                       y=None, state_final=None, want_final_state=True, stream=None):
    """Causal depthwise convolution over time, y_t = act(bias + sum_w weight[:,w]
    x_{t-W+1+w}).  Returns ``(y, state_final)``.

    ``x`` [B,L,D] fp32 or bf16; its rows may be a slice of a wider tensor.
    ``weight`` fp32 [D,W] with W in 2..8, ``bias`` fp32 [D].  ``activation``:
    "silu" | "none".  ``state0`` and ``state_final`` [B,W-1,D] in x's dtype are
    the W-1 inputs before the first and up to the last token; they may be one
    tensor (with L = 1 that is one decode step in place).  ``lengths`` int32 [B]
    are the real tokens of a padded batch: the rows of ``y`` behind them are
    left as they are (zero when ``y`` is made here)."""
    shape, dtype = x.shape, x.dtype
    B, L, D = shape
    W = weight.shape[-1]
    if max(B, L, D, W) > _INT_MAX:
        raise _too_large(B, L, D, W)
    xs = D if x.is_contiguous() else _row_stride(x, shape, dtype, "x")
    w = _param(weight, (D, W), "weight")
    bi = None if bias is None else _param(bias, (D,), "bias")
    n = None if lengths is None else _lengths_ptr(lengths, B)
    state = (B, W - 1, D)
    s0 = None if state0 is None else _conv_state(state0, state, dtype)
    s1 = None if state_final is None else _conv_state(state_final, state, dtype)
    dev = _device_of(x, weight, bias, state0, lengths, y, state_final)
    if y is None:
        y = _new(shape, dtype, x.device, stream, lengths is not None)
    if state_final is None and want_final_state:
        state_final = _new(state, dtype, x.device, stream)
        s1 = state_final.data_ptr()
    status = _native.load().la_causal_conv_fwd(
        x.data_ptr(), xs, DTYPE[dtype], B, L, D, W, w, bi, ACT[activation], n, s0, y.data_ptr(),
        _row_stride(y, shape, dtype, "y"), s1,
        _current_stream(dev) if stream is None else stream.cuda_stream)
    if status:
        _check(status)
    return y, state_final


def la_selective_scan_fwd_workspace_bytes(B, L, D, N, groups=1) -> int:
    return int(_native.load().la_selective_scan_fwd_workspace_bytes(B, L, D, N, groups))


def la_selective_scan_fwd(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, dt_softplus=True,
                          h0=None, lengths=None, y=None, h_final=None, want_final_state=True,
                          workspace=None, segments=True, stream=None):
    """Selective state space scan h = exp(delta A) h + delta B x, y = (C h + D x)
    silu(z), delta = softplus(dt + dt_bias).  Returns ``(y, h_final)``.

    ``x``, ``dt``, ``z`` [B,L,channels] and ``Bm``, ``Cm`` [B,L,N] or
    [B,L,groups,N], all fp32 or all bf16; each may be a slice of a wider
    tensor.  ``A`` fp32 [channels,N] (N <= 256), ``D`` and ``dt_bias`` fp32
    [channels].  ``h0`` and ``h_final`` fp32 [B,channels,N] may be one tensor
    (with L = 1 that is one decode step in place).  ``lengths`` int32 [B] are
    the real tokens of a padded batch: the rows of ``y`` behind them are left
    as they are (zero when ``y`` is made here).  With ``segments`` (the
    default) a workspace lets a long sequence run as several segments side by
    side."""
    shape, dtype = x.shape, x.dtype
    B, L, ch = shape
    N = A.shape[-1]
    bc = Bm.shape
    G = bc[2] if len(bc) == 4 else 1
    if bc != ((B, L, G, N) if len(bc) == 4 else (B, L, N)):
        raise ValueError("Bm must be [B,L,N] or [B,L,groups,N]")
    if max(B, L, ch, N, G) > _INT_MAX:
        raise _too_large(B, L, ch, N, G)
    xs = _row_stride(x, shape, dtype, "x")
    ds = _row_stride(dt, shape, dtype, "dt")
    zs = 0 if z is None else _row_stride(z, shape, dtype, "z")
    bs = _row_stride(Bm, bc, dtype, "Bm")
    cs = _row_stride(Cm, bc, dtype, "Cm")
    per, state = (ch,), (B, ch, N)
    Ap = _param(A, (ch, N), "A")
    Dp = None if D is None else _param(D, per, "D")
    bias = None if dt_bias is None else _param(dt_bias, per, "dt_bias")
    h0p = None if h0 is None else _param(h0, state, "h0")
    hfp = None if h_final is None else _param(h_final, state, "h_final")
    n = None if lengths is None else _lengths_ptr(lengths, B)
    dev = _device_of(x, dt, z, Bm, Cm, A, D, dt_bias, h0, lengths, y, h_final, workspace)
    if y is None:
        y = _new(shape, dtype, x.device, stream, lengths is not None)
    if h_final is None and want_final_state:
        h_final = _new(state, torch.float32, x.device, stream)
        hfp = h_final.data_ptr()
    lib = _native.load()
    ws = ws_bytes = 0
    if workspace is None and segments and L > 1:
        workspace = _workspace(lib.la_selective_scan_fwd_workspace_bytes(B, L, ch, N, G),
                               x.device, stream)
    if workspace is not None:
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    status = lib.la_selective_scan_fwd(
        x.data_ptr(), xs, dt.data_ptr(), ds, None if z is None else z.data_ptr(), zs,
        Bm.data_ptr(), bs, Cm.data_ptr(), cs, DTYPE[dtype], B, L, ch, N, G, Ap, bias,
        dt_softplus, Dp, h0p, n, y.data_ptr(), _row_stride(y, shape, dtype, "y"), hfp, ws,
        ws_bytes, _current_stream(dev) if stream is None else stream.cuda_stream)
    if status:
        _check(status)
    return y, h_final


def _head_param(t, H, d):
    """A gated norm's weight or bias: its address and the heads it is given for."""
    n = t.numel()
    if t.dtype != torch.float32 or not t.is_contiguous() or (n != d and n != H * d):
        raise ValueError("weight and bias must be contiguous fp32 [d] or [H*d]")
    return t.data_ptr(), 1 if n == d else H


def la_gated_norm_fwd(x, gate=None, weight=None, bias=None, norm="rms", activation="silu",
                      gate_first=False, eps=1e-5, y=None, stream=None):
    """Norm over the last axis of ``x`` [B,H,L,d] times ``weight`` and act(gate),
    written token major as [B,L,H*d] for the output projection.  Returns ``y``.

    ``x`` fp32 or bf16 with any strides whose last is 1: O of the attention
    calls as it is, or a permuted view of a token-major tensor.  ``gate``
    [B,L,H*d]; ``weight`` and ``bias`` fp32 [d] (shared by the heads) or [H*d].
    ``norm``: "rms" | "layer"; ``activation``: "silu" | "sigmoid" | "none";
    ``gate_first`` gates x before its norm instead of after it.  ``y`` may be
    ``gate``."""
    B, H, L, d = x.shape
    dtype = x.dtype
    xb, xh, xt, x1 = x.stride()
    if x1 != 1 and d > 1 and x.numel() > 0:
        raise ValueError("the last axis of x must be contiguous")
    if max(B, H, L, d) > _INT_MAX:
        raise _too_large(B, H, L, d)
    width = H * d
    shape = (B, L, width)
    heads = 1
    w = b = None
    if weight is not None:
        w, heads = _head_param(weight, H, d)
    if bias is not None:
        b, heads = _head_param(bias, H, d)
        if weight is not None and weight.numel() != bias.numel():
            raise ValueError("weight and bias must have one shape")
    gs = 0 if gate is None else _row_stride(gate, shape, dtype, "gate")
    dev = _device_of(x, gate, weight, bias, y)
    if y is None:
        y = _new(shape, dtype, x.device, stream)
    status = _native.load().la_gated_norm_fwd(
        x.data_ptr(), xb, xh, xt, None if gate is None else gate.data_ptr(), gs, DTYPE[dtype],
        B, H, L, d, NORM[norm], ACT[activation], gate_first, w, b, heads, eps, y.data_ptr(),
        _row_stride(y, shape, dtype, "y"),
        _current_stream(dev) if stream is None else stream.cuda_stream)
    if status:
        _check(status)
    return y


def _same(t, shape, dtype):
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
        raise ValueError("x, residual and the outputs must be contiguous and of one shape, y in "
                         "x's dtype and residual_out in residual's")
    return t.data_ptr()


def la_residual_norm_fwd(x, residual=None, weight=None, bias=None, post_weight=None, scale=None,
                         alpha=1.0, norm="rms", eps=1e-5, y=None, residual_out=None,
                         residual_dtype=None, stream=None):
    """The step between two blocks: r = residual + alpha scale post(x) with
    post(x) = norm(x) post_weight (x itself without ``post_weight``), then
    y = norm(r) weight + bias.  Returns ``(y, residual_out)`` with residual_out
    = r.

    ``x`` [...,D] contiguous, fp32 or bf16; ``residual`` the same shape, in x's
    dtype or fp32 (None: zero; ``residual_dtype`` then chooses residual_out's,
    x's by default).  The parameters are fp32 [D].  ``y`` may be ``x`` and
    ``residual_out`` may be ``residual``."""
    shape, dtype = x.shape, x.dtype
    D = shape[-1]
    if D > _INT_MAX:
        raise _too_large(D)
    rd = residual.dtype if residual is not None else \
        residual_out.dtype if residual_out is not None else residual_dtype or dtype
    per = (D,)
    pw = None if post_weight is None else _param(post_weight, per, "post_weight")
    sc = None if scale is None else _param(scale, per, "scale")
    w = None if weight is None else _param(weight, per, "weight")
    bi = None if bias is None else _param(bias, per, "bias")
    xp = _same(x, shape, dtype)
    rp = None if residual is None else _same(residual, shape, rd)
    yp = None if y is None else _same(y, shape, dtype)
    op = None if residual_out is None else _same(residual_out, shape, rd)
    dev = _device_of(x, residual, weight, bias, post_weight, scale, y, residual_out)
    if y is None:
        y = _new(shape, dtype, x.device, stream)
        yp = y.data_ptr()
    if residual_out is None:
        residual_out = _new(shape, rd, x.device, stream)
        op = residual_out.data_ptr()
    status = _native.load().la_residual_norm_fwd(
        xp, DTYPE[dtype], rp, DTYPE[rd], x.numel() // D if D else 0, D, pw, sc, alpha, w, bi,
        NORM[norm], eps, yp, op, _current_stream(dev) if stream is None else stream.cuda_stream)
    if status:
        _check(status)
    return y, residual_out


# ---------------------------------------------------------------- training pass
def la_rotary_frequencies(rotary_dim, base=10000.0, scaling="plain", factor=1.0,
                          trained_length=0.0, fast=32.0, slow=1.0):
    """Rotary frequencies ``(inv_freq, scale)``: fp32 [rotary_dim/2] in host memory
    (``.cuda()`` them once) and the factor of q and k.  ``scaling``: "plain" |
    "linear" (positions interpolated by ``factor``) | "ntk" (a larger base) |
    "yarn" (pairs of fewer than ``slow`` turns over ``trained_length`` interpolated,
    those of more than ``fast`` left, a blend linear in the pair's index between, from and
    to whole pairs: what checkpoints with this scaling are trained with)."""
    if rotary_dim > _INT_MAX:
        raise _too_large(rotary_dim)
    inv_freq = torch.empty(max(rotary_dim // 2, 0), dtype=torch.float32)
    scale = torch.empty(1, dtype=torch.float32)
    _check(_native.load().la_rotary_frequencies(
        rotary_dim, base, ROTARY[scaling], factor, trained_length, fast, slow,
        inv_freq.data_ptr(), scale.data_ptr()))
    return inv_freq, scale.item()


def _like(t, stream):
    """A tensor like ``t`` (contiguous, its shape and dtype) on the call's stream: with no stream
    given, half of the host's time that ``_new`` takes."""
    if stream is None:
        return torch.empty_like(t, memory_format=torch.contiguous_format)
    return _new(t.shape, t.dtype, t.device, stream)


def _scratch(nbytes, t, stream):
    """A call's workspace (see ``_workspace``), made from one of its tensors."""
    if not nbytes:
        return None
    if stream is None:
        return t.new_empty(-(-nbytes // t.element_size()))
    return _workspace(nbytes, t.device, stream)


def _int32(t, shape, what):
    if t.dtype != torch.int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous int32 {list(shape)}")
    return t.data_ptr()


def _heads(t, shape, dtype, what):
    """Address and strides of ``t`` = [B,H,L,d] whose last axis is contiguous."""
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{what} must be {dtype} {list(shape)}")
    b, h, n, one = t.stride()
    if one != 1 and shape[3] > 1 and t.numel() > 0:
        raise ValueError(f"the last axis of {what} must be contiguous")
    return t.data_ptr(), b, h, n


_NO_HEADS = (None, 0, 0, 0)


def _rotary(call, q, k, inv_freq, positions, offsets, lengths, interleaved, scale, q_out, k_out,
            stream):
    shape, dtype = q.shape, q.dtype
    B, H, L, d = shape
    Hk, ka, k_shape = 0, _NO_HEADS, None
    qa = _heads(q, shape, dtype, "q")
    if k is not None:
        k_shape = k.shape
        if len(k_shape) != 4 or k_shape[0] != B or k_shape[2] != L or k_shape[3] != d:
            raise ValueError("q and k must agree in [B,.,L,d]")
        Hk = k_shape[1]
        ka = _heads(k, k_shape, dtype, "k")
    elif k_out is not None:
        raise ValueError("k_out without k")
    if max(B, H, Hk, L, d) > _INT_MAX:
        raise _too_large(B, H, Hk, L, d)
    pairs = inv_freq.numel()
    f = _param(inv_freq, (pairs,), "inv_freq")
    ps = None if positions is None else _int32(positions, (B, L), "positions")
    of = None if offsets is None else _int32(offsets, (B,), "offsets")
    n = None if lengths is None else _int32(lengths, (B,), "lengths")
    dev = _device_of(q, k, inv_freq, positions, offsets, lengths, q_out, k_out)
    if q_out is None:
        q_out = _new(shape, dtype, q.device, stream, lengths is not None)
    qo = _heads(q_out, shape, dtype, "q_out")
    ko = _NO_HEADS
    if k is not None:
        if k_out is None:
            k_out = _new(k_shape, dtype, q.device, stream, lengths is not None)
        ko = _heads(k_out, k_shape, dtype, "k_out")
    status = call(
        qa[0], qa[1], qa[2], qa[3], H, ka[0], ka[1], ka[2], ka[3], Hk, DTYPE[dtype], B, L, d,
        2 * pairs, interleaved, f, scale, ps, of, n, qo[0], qo[1], qo[2], qo[3], ko[0], ko[1],
        ko[2], ko[3], _current_stream(dev) if stream is None else stream.cuda_stream)
    if status:
        _check(status)
    return q_out, k_out


def la_rotary_fwd(q, k, inv_freq, positions=None, offsets=None, lengths=None, interleaved=False,
                  scale=1.0, q_out=None, k_out=None, stream=None):
    """Rotary positions of ``q`` [B,H,L,d] and ``k`` [B,H_k,L,d] (or None) in one
    call.  Returns ``(q_out, k_out)``, [B,H,L,d] as ``la_chunk_fwd`` reads them
    unless given.

    ``q``, ``k`` and the outputs are fp32 or bf16 with any strides whose last is 1: a
    permuted view of a projection's token-major output as it is.  ``inv_freq``
    fp32 [r/2] (``la_rotary_frequencies``) turns the first r values of a head, in
    pairs of neighbours if ``interleaved``, else (i, i + r/2).  Token t of sequence
    b has position ``offsets[b] + t``, or ``offsets[b] + positions[b,t]`` (int32 [B] and
    [B,L]).  ``lengths`` int32 [B]: the tokens behind them are left as they are in the
    outputs (zero where these are made here).  ``q_out`` may be ``q``, ``k_out`` ``k``."""
    return _rotary(_native.load().la_rotary_fwd, q, k, inv_freq, positions, offsets, lengths, interleaved,
                   scale, q_out, k_out, stream)


def la_rotary_bwd(dq, dk, inv_freq, positions=None, offsets=None, lengths=None,
                  interleaved=False, scale=1.0, q_out=None, k_out=None, stream=None):
    """Backward pass of ``la_rotary_fwd``: the gradients of its outputs to those of
    its inputs, of the same arguments.  ``q_out`` and ``k_out`` may be views of a
    projection's gradient.  Returns ``(q_out, k_out)``."""
    return _rotary(_native.load().la_rotary_bwd, dq, dk, inv_freq, positions, offsets, lengths, interleaved,
                   scale, q_out, k_out, stream)


def la_chunk_bwd_workspace_bytes(B, H, L, d_k, d_v, chunk=64, dtype=torch.bfloat16) -> int:
    if max(B, H, L, d_k, d_v, chunk) > _INT_MAX:
        raise _too_large(B, H, L, d_k, d_v, chunk)
    return int(_native.load().la_chunk_bwd_workspace_bytes(B, H, L, d_k, d_v, chunk,
                                                           DTYPE[dtype]))


def la_chunk_bwd_workspace_bytes_for(B, H, L, d_k, d_v, chunk=64, dtype=torch.bfloat16,
                                     decay_kind="none", ddecay=False, dS0=False) -> int:
    """What one call needs, with the feature map set now: ``ddecay`` and ``dS0`` whether those
    gradients are formed.  (``la_chunk_bwd_workspace_bytes`` is enough for any call.)"""
    if max(B, H, L, d_k, d_v, chunk) > _INT_MAX:
        raise _too_large(B, H, L, d_k, d_v, chunk)
    return int(_native.load().la_chunk_bwd_workspace_bytes_for(
        B, H, L, d_k, d_v, chunk, DTYPE[dtype], DECAY[decay_kind], ddecay, dS0))


def _dense(t, shape, dtype, what):
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous {dtype} {list(shape)}")
    return t.data_ptr()


def la_chunk_bwd(q, k, v, dO, chunk=64, decay_kind="none", decay=None, S0=None, dS_final=None,
                 dq=None, dk=None, dv=None, ddecay=None, dS0=None, want_decay_grad=True,
                 want_state_grad=None, workspace=None, stream=None):
    """Backward pass of ``la_chunk_fwd`` (with the feature map set now): from ``dO``,
    the gradient of O, ``dS_final``, that of S_final (None: zero), and the forward
    call's arguments.  Returns ``(dq, dk, dv, ddecay, dS0)``.

    ``ddecay`` has ``decay``'s shape: the gradient of log gamma [H], log alpha or the
    gate logits [B,H,L]; None without a decay or without ``want_decay_grad``.  ``dS0``
    is formed with ``S0`` unless ``want_state_grad`` says otherwise.  With bf16 tensors
    both cost about twice the work: their products keep 24 bits."""
    shape, dtype = q.shape, q.dtype
    B, H, L, d_k = shape
    d_v = v.shape[-1]
    if max(B, H, L, d_k, d_v, chunk) > _INT_MAX:
        raise _too_large(B, H, L, d_k, d_v, chunk)
    v_shape, state, f32 = (B, H, L, d_v), (B, H, d_k, d_v), torch.float32
    kind = DECAY[decay_kind]
    if (decay is None) != (kind == 0):
        raise ValueError("decay goes with its decay_kind")
    decay_shape = (H,) if kind == 1 else (B, H, L)
    qp, kp = _dense(q, shape, dtype, "q"), _dense(k, shape, dtype, "k")
    vp, dOp = _dense(v, v_shape, dtype, "v"), _dense(dO, v_shape, dtype, "dO")
    dp = None if decay is None else _dense(decay, decay_shape, f32, "decay")
    s0 = None if S0 is None else _dense(S0, state, f32, "S0")
    sf = None if dS_final is None else _dense(dS_final, state, f32, "dS_final")
    dev = _device_of(q, k, v, dO, decay, S0, dS_final, dq, dk, dv, ddecay, dS0, workspace)
    dq = _like(q, stream) if dq is None else dq
    dk = _like(k, stream) if dk is None else dk
    dv = _like(v, stream) if dv is None else dv
    if ddecay is not None and decay is None:
        raise ValueError("ddecay without a decay")
    if ddecay is None and want_decay_grad and decay is not None:
        ddecay = _like(decay, stream)
    if dS0 is None and (S0 is not None if want_state_grad is None else want_state_grad):
        dS0 = _new(state, f32, q.device, stream)
    lib = _native.load()
    ws = ws_bytes = 0
    if workspace is None:
        workspace = _scratch(lib.la_chunk_bwd_workspace_bytes_for(
            B, H, L, d_k, d_v, chunk, DTYPE[dtype], kind, ddecay is not None, dS0 is not None), q,
            stream)
    if workspace is not None:
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    status = lib.la_chunk_bwd(
        qp, kp, vp, DTYPE[dtype], B, H, L, d_k, d_v, chunk, kind, dp, s0, dOp, sf,
        _dense(dq, shape, dtype, "dq"), _dense(dk, shape, dtype, "dk"),
        _dense(dv, v_shape, dtype, "dv"),
        None if ddecay is None else _dense(ddecay, decay_shape, f32, "ddecay"),
        None if dS0 is None else _dense(dS0, state, f32, "dS0"), ws, ws_bytes,
        _current_stream(dev) if stream is None else stream.cuda_stream)
    if status:
        _check(status)
    return dq, dk, dv, ddecay, dS0


def la_gated_norm_bwd_workspace_bytes(B, H, L, d, weight_heads=1) -> int:
    if max(B, H, L, d, weight_heads) > _INT_MAX:
        raise _too_large(B, H, L, d, weight_heads)
    return int(_native.load().la_gated_norm_bwd_workspace_bytes(B, H, L, d, weight_heads))


def la_gated_norm_bwd(dy, x, gate=None, weight=None, bias=None, norm="rms", activation="silu",
                      gate_first=False, eps=1e-5, dx=None, dgate=None, dweight=None, dbias=None,
                      want_param_grads=True, workspace=None, stream=None):
    """Backward pass of ``la_gated_norm_fwd``: from ``dy`` [B,L,H*d], the gradient of
    its output, and its arguments.  Returns ``(dx, dgate, dweight, dbias)``.

    ``dx`` [B,H,L,d] in x's dtype (any strides whose last is 1; made contiguous),
    ``dgate`` [B,L,H*d], ``dweight`` and ``dbias`` fp32 of the parameters' shapes; None
    for what is not there, and for the parameters' without ``want_param_grads``.  ``dx``
    may be ``x``, ``dgate`` ``gate`` or ``dy``."""
    B, H, L, d = x.shape
    dtype = x.dtype
    if max(B, H, L, d) > _INT_MAX:
        raise _too_large(B, H, L, d)
    width = H * d
    shape = (B, L, width)
    heads = 1
    w = b = None
    if weight is not None:
        w, heads = _head_param(weight, H, d)
    if bias is not None:
        b, heads = _head_param(bias, H, d)
        if weight is not None and weight.numel() != bias.numel():
            raise ValueError("weight and bias must have one shape")
    if gate is None and dgate is not None:
        raise ValueError("dgate without a gate")
    xa = _heads(x, x.shape, dtype, "x")
    dys = _row_stride(dy, shape, dtype, "dy")
    gs = 0 if gate is None else _row_stride(gate, shape, dtype, "gate")
    dev = _device_of(x, dy, gate, weight, bias, dx, dgate, dweight, dbias, workspace)
    for g, p, what in ((dweight, weight, "dweight"), (dbias, bias, "dbias")):
        if g is not None and (p is None or g.shape != p.shape):
            raise ValueError(f"{what} must have its parameter's shape")
    if dx is None:
        dx = _like(x, stream)
    if gate is not None and dgate is None:
        dgate = _like(gate, stream)
    if want_param_grads:
        if weight is not None and dweight is None:
            dweight = _like(weight, stream)
        if bias is not None and dbias is None:
            dbias = _like(bias, stream)
    lib = _native.load()
    ws = ws_bytes = 0
    if workspace is None and (dweight is not None or dbias is not None):
        workspace = _scratch(lib.la_gated_norm_bwd_workspace_bytes(B, H, L, d, heads), x, stream)
    if workspace is not None:
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    status = lib.la_gated_norm_bwd(
        dy.data_ptr(), dys, *xa, None if gate is None else gate.data_ptr(), gs, DTYPE[dtype], B, H,
        L, d, NORM[norm], ACT[activation], gate_first, w, b, heads, eps,
        *_heads(dx, x.shape, dtype, "dx"), None if gate is None else dgate.data_ptr(),
        0 if gate is None else _row_stride(dgate, shape, dtype, "dgate"),
        None if dweight is None else _param(dweight, dweight.shape, "dweight"),
        None if dbias is None else _param(dbias, dbias.shape, "dbias"), ws, ws_bytes,
        _current_stream(dev) if stream is None else stream.cuda_stream)
    if status:
        _check(status)
    return dx, dgate, dweight, dbias


def la_residual_norm_bwd_workspace_bytes(rows, D) -> int:
    if D > _INT_MAX:
        raise _too_large(D)
    return int(_native.load().la_residual_norm_bwd_workspace_bytes(rows, D))


def la_residual_norm_bwd(dy, r, weight=None, dr=None, x=None, post_weight=None, scale=None,
                         alpha=1.0, norm="rms", eps=1e-5, dx=None, dresidual=None,
                         want_dresidual=True, want_param_grads=True, want_dbias=False,
                         workspace=None, stream=None):
    """Backward pass of ``la_residual_norm_fwd``: from ``dy``, the gradient of its y,
    ``r``, the residual_out that it wrote, and ``dr``, the gradient of that (None:
    zero).  Returns ``(dx, dresidual, dweight, dbias, dpost_weight, dscale)``.

    ``dy``, ``x`` and ``dx`` [...,D] fp32 or bf16, ``r``, ``dr`` and ``dresidual`` in
    that dtype or fp32, all contiguous; ``x`` is needed with ``post_weight`` or
    ``scale``.  The parameters' gradients are fp32 [D], None for what is not there
    (``dbias`` is formed if ``want_dbias``: the bias itself is not needed).  ``dx`` may
    be ``dy`` or ``x``, ``dresidual`` may be ``dr``.  By itself, with ``weight`` and
    ``want_dbias``, this is a layer norm's backward pass."""
    shape, dtype = dy.shape, dy.dtype
    D = shape[-1]
    if D > _INT_MAX:
        raise _too_large(D)
    rd = r.dtype
    per = (D,)
    w = None if weight is None else _param(weight, per, "weight")
    pw = None if post_weight is None else _param(post_weight, per, "post_weight")
    sc = None if scale is None else _param(scale, per, "scale")
    yp, rp = _same(dy, shape, dtype), _same(r, shape, rd)
    drp = None if dr is None else _same(dr, shape, rd)
    xp = None if x is None else _same(x, shape, dtype)
    dev = _device_of(dy, r, dr, x, weight, post_weight, scale, dx, dresidual, workspace)
    dx = _like(dy, stream) if dx is None else dx
    if dresidual is None and want_dresidual:
        dresidual = _like(r, stream)
    grads = [None] * 4  # of weight, bias, post_weight, scale
    if want_param_grads:
        grads = [_like(weight, stream) if w else None, None,
                 _like(post_weight, stream) if pw else None, _like(scale, stream) if sc else None]
    if want_dbias:
        grads[1] = _like(weight, stream) if w else _new(per, torch.float32, dy.device, stream)
    rows = dy.numel() // D if D else 0
    lib = _native.load()
    ws = ws_bytes = 0
    if workspace is None and (want_dbias or want_param_grads and (w or pw or sc)):
        workspace = _scratch(lib.la_residual_norm_bwd_workspace_bytes(rows, D), dy, stream)
    if workspace is not None:
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    status = lib.la_residual_norm_bwd(
        yp, DTYPE[dtype], rp, drp, DTYPE[rd], xp, rows, D, pw, sc, alpha, w, NORM[norm], eps,
        _same(dx, shape, dtype), None if dresidual is None else _same(dresidual, shape, rd),
        *[None if g is None else g.data_ptr() for g in grads], ws, ws_bytes,
        _current_stream(dev) if stream is None else stream.cuda_stream)
    if status:
        _check(status)
    return (dx, dresidual, *grads)


def la_device_status(stream=None) -> None:
    """Synchronise and raise LAError if a kernel's bounded wait timed out."""
    _check(_native.load().la_device_status(_stream(stream)))


def la_selftest_wait_timeout(spin_limit: int = 1000, stream=None) -> int:
    """Run the timeout self-test kernel; returns the status it reports."""
    lib = _native.load()
    return lib.la_selftest_wait_timeout(spin_limit, _stream(stream))


def la_last_error() -> str:
    return _native.load().la_last_error().decode()
