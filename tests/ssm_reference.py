"""The state space block's operators in 64 bits, token by token from their
formulas, each with an elementwise bound on what an fp32 evaluation may be off.

Every function returns (values, bound) pairs as float64 arrays.  The bounds
count roundings: U = 2^-24 is half an fp32 step relative to a value, and an
output of type t adds half a step of t, ``half_step(t) * |value|``.  Errors of
the pieces: a sum of k products errs by at most (k + 1) U times the sum of the
magnitudes; exp2 on the special-function unit and a reciprocal err by 2^-22
and 2^-23 relative; the argument of an exponential is rounded (and scaled by
log2 e), which moves exp(a) by 3 U |a| relative.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
SFU = 2.0 ** -22
TINY = 2.0 ** -126


def half_step(dtype: str) -> float:
    return {"bf16": 2.0 ** -8, "f32": U}[dtype]


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def act(kind, x):
    """Value, error of its evaluation, and a bound of |act'|.  fp32 has no
    normal numbers below 2^-126: where e^-x passes 2^126 the sigmoid is 0, which
    is off by up to 2^-126, and x sigmoid(x) by up to |x| 2^-126."""
    rel = 3 * U * np.abs(x) + SFU + 4 * U
    s = sigmoid(x)
    if kind == "silu":
        return x * s, np.abs(x) * (s * rel + TINY), 1.1
    if kind == "sigmoid":
        return s, s * rel + TINY, 0.25
    return x, 0.0 * x, 1.0


def causal_conv(x, weight, bias, activation, state0, lengths, dtype):
    """((y, bound), state_final).  Rows of y behind a length are NaN (not to be compared)."""
    x, weight, bias, state0 = f64(x), f64(weight), f64(bias), f64(state0)
    B, L, D = x.shape
    W = weight.shape[1]
    n = np.full(B, L) if lengths is None else np.clip(lengths.cpu().numpy(), 0, L)
    y = np.full((B, L, D), np.nan)
    tol = np.zeros((B, L, D))
    last = np.zeros((B, W - 1, D))
    for b in range(B):
        past = np.zeros((W - 1, D)) if state0 is None else state0[b]
        xs = np.concatenate([past, x[b, :n[b]]])
        last[b] = xs[n[b]:]
        for t in range(n[b]):
            terms = xs[t:t + W].T * weight
            s = terms.sum(1) + (0 if bias is None else bias)
            m = np.abs(terms).sum(1) + (0 if bias is None else np.abs(bias))
            y[b, t], err, slope = act(activation, s)
            tol[b, t] = slope * (W + 2) * U * m + err + half_step(dtype) * np.abs(y[b, t])
    return (y, tol), last


def selective_scan(x, dt, A, Bm, Cm, D, z, dt_bias, softplus, h0, lengths, dtype):
    """((y, bound), (h_final, bound)).  Rows of y behind a length are NaN."""
    x, dt, A, Bm, Cm, D, z, dt_bias, h0 = map(f64, (x, dt, A, Bm, Cm, D, z, dt_bias, h0))
    B, L, ch = x.shape
    N = A.shape[1]
    Bm, Cm = (t.reshape(B, L, -1, N) for t in (Bm, Cm))
    G = Bm.shape[2]
    of = np.arange(ch) // (ch // G)  # a channel's group
    n = np.full(B, L) if lengths is None else np.clip(lengths.cpu().numpy(), 0, L)
    y = np.full((B, L, ch), np.nan)
    ytol = np.zeros((B, L, ch))
    hf = np.zeros((B, ch, N))
    htol = np.zeros((B, ch, N))
    skip = np.zeros(ch) if D is None else D
    for b in range(B):
        h = np.zeros((ch, N)) if h0 is None else h0[b].copy()
        H, E = np.abs(h), np.zeros((ch, N))  # magnitudes, and the error so far
        for t in range(n[b]):
            v = dt[b, t] + (0 if dt_bias is None else dt_bias)
            delta, rel = v, U + np.zeros(ch)
            if softplus:
                # v errs by U |v|, the logistic slope over the value is below 1;
                # exp, reciprocal, series and the final sum below 2^-21
                delta, rel = np.logaddexp(0, v), U * np.abs(v) + 8 * U
            size = np.abs(delta)[:, None] * np.abs(A)
            a = np.exp(delta[:, None] * A)
            w = (delta * x[b, t])[:, None] * Bm[b, t][of]
            h = a * h + w
            H = a * H + np.abs(w)
            # the decay errs by SFU, by 3 U and by delta's own error times its
            # exponent; the write by delta's error and three roundings; the sum by one
            E = a * E + H * (SFU + 6 * U + size * (3 * U) + (1 + size) * rel[:, None])
            c = Cm[b, t][of]
            s = (c * h).sum(1) + skip * x[b, t]
            m = (np.abs(c) * H).sum(1) + np.abs(skip * x[b, t])
            e = (np.abs(c) * E).sum(1) + (N + 3) * U * m
            g, gerr = (1.0, 0.0) if z is None else act("silu", z[b, t])[:2]
            y[b, t] = s * g
            ytol[b, t] = (e * np.abs(g) + (np.abs(s) + e) * gerr
                          + np.abs(y[b, t]) * (U + half_step(dtype)))
        hf[b], htol[b] = h, E
    return (y, ytol), (hf, htol)


def _norm(v, e, kind, eps):
    """norm(v) over the last axis, and its error where v errs by e: a sum over
    d values is taken in runs of at most d / 32 values and five to ten halvings."""
    d = v.shape[-1]
    k = d / 32 + 12
    if kind == "layer":
        mean = v.mean(-1, keepdims=True)
        e = e + k * U * np.abs(v).mean(-1, keepdims=True) + e.mean(-1, keepdims=True)
        v = v - mean
        e = e + U * np.abs(v)
    q = (v * v).mean(-1, keepdims=True)
    dq = k * U * q + 2 * (np.abs(v) * e).mean(-1, keepdims=True) + (e * e).mean(-1, keepdims=True)
    r = 1 / np.sqrt(q + eps)
    rel = 0.5 * dq / (q + eps) + 4 * U
    return v * r, e * r + np.abs(v * r) * (rel + 2 * U)


def gated_norm(x, gate, weight, bias, norm, activation, gate_first, eps, dtype):
    """(y, bound) in the [B,L,H*d] layout."""
    x, gate, weight, bias = map(f64, (x, gate, weight, bias))
    B, H, L, d = x.shape
    v = x.transpose(0, 2, 1, 3)
    e = np.zeros_like(v)
    g, gerr = 1.0, 0.0
    if gate is not None:
        g, gerr, _ = act(activation, gate.reshape(B, L, H, d))
    shape = lambda w: w if w is None or w.size == d else w.reshape(H, d)  # noqa: E731
    if gate_first:
        v, e = v * g, np.abs(v) * gerr + U * np.abs(v * g)
    v, e = _norm(v, e, norm, eps)
    if weight is not None:
        v, e = v * shape(weight), e * np.abs(shape(weight)) + U * np.abs(v * shape(weight))
    if bias is not None:
        v = v + shape(bias)
        e = e + U * np.abs(v)
    if not gate_first:
        v, e = v * g, e * np.abs(g) + (np.abs(v) + e) * gerr + U * np.abs(v * g)
    e = e + half_step(dtype) * np.abs(v)
    return v.reshape(B, L, H * d), e.reshape(B, L, H * d)


def residual_norm(x, residual, post_weight, scale, alpha, weight, bias, norm, eps, dtype,
                  res_dtype):
    """((y, bound), (residual_out, bound))."""
    x, residual, post_weight, scale, weight, bias = map(
        f64, (x, residual, post_weight, scale, weight, bias))
    alpha = float(np.float32(alpha))
    u, e = x, np.zeros_like(x)
    if post_weight is not None:
        u, e = _norm(u, e, norm, eps)
        u, e = u * post_weight, e * np.abs(post_weight) + U * np.abs(u * post_weight)
    if scale is not None:
        u, e = u * scale, e * np.abs(scale) + U * np.abs(u * scale)
    u, e = alpha * u, abs(alpha) * e + U * np.abs(alpha * u)
    r = u if residual is None else residual + u
    e = e + U * np.abs(r)
    v, ev = _norm(r, e, norm, eps)
    if weight is not None:
        v, ev = v * weight, ev * np.abs(weight) + U * np.abs(v * weight)
    if bias is not None:
        v = v + bias
        ev = ev + U * np.abs(v)
    return (v, ev + half_step(dtype) * np.abs(v)), (r, e + half_step(res_dtype) * np.abs(r))


def check(got, ref, what, live=None):
    """Every element within its bound; ``live`` selects the rows to compare."""
    val, tol = ref
    got = f64(got)
    assert got.shape == val.shape, (what, got.shape, val.shape)
    if live is not None:
        got, val, tol = got[live], val[live], tol[live]
    assert np.isfinite(got).all() == np.isfinite(val).all(), what
    # 1e-37: below it fp32 runs out of normal numbers
    over = np.abs(got - val) - (tol + 1e-37)
    worst = np.unravel_index(np.argmax(over), over.shape) if over.size else None
    assert over.size == 0 or over.max() <= 0, \
        f"{what}: at {worst} got {got[worst]!r}, want {val[worst]!r} within {tol[worst]:.3e}"
