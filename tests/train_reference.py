"""The operators of a layer's training pass in 64 bits, from their formulas, each with an elementwise
bound on what the kernels' arithmetic may be off.

Every function returns (values, bound) pairs as float64 arrays (``ssm_reference.check`` compares).
The bounds count roundings as there: U = 2^-24 is half an fp32 step relative to a value, an output of
type t adds half a step of t.  Where an output is a sum of products its bound is a number of
roundings times the sum of the products' magnitudes, which runs through the same recurrence with
every factor's absolute value in its place.

The attention's counts.  With bf16 tensors a product takes operands that were rounded to bf16 (2^-8
each): the score, or the state and the decayed key or query that entered it; with phi = elu + 1 also
phi's value of the query and of the key.  That is two roundings at most, with elu + 1 four, and
their products err by a little more than the sum.  Products that keep 24 bits,
and all of fp32's, err by fp32 roundings: three planes leave 2^-24 of an operand, the tensor cores
cut 2^-23 of a sum off for every 16 products (at most 8 times in a row of 128), an exponential or a
decay's factor errs by 2^-21 and a product holds at most four of them, and a state takes three
roundings for every chunk of at least 32 tokens that it passes.
"""
from __future__ import annotations

import numpy as np

from tests.ssm_reference import SFU, TINY, U, act, f64, half_step, sigmoid

BF16 = 2.0 ** -8


# ---------------------------------------------------------------- rotary positions
def rotary(x, inv_freq, positions, scale, interleaved, backward, dtype):
    """(y, bound) of [B,H,L,d]; positions [B,L] as int64.  The angle is exact to position * 2^-64
    turns; sine and cosine err by 2^-22 (their argument's rounding, six coefficients'), the scaled
    factors and the two products by U each."""
    x, f = f64(x), f64(inv_freq)
    pos = positions.numpy().astype(np.float64)
    angle = pos[..., None] * f
    angle = angle if not backward else -angle
    scale = float(np.float32(scale))
    c, s = (scale * g(angle)[:, None] for g in (np.cos, np.sin))
    r = 2 * f.size
    y, tol = x.copy(), np.zeros_like(x)
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        places = (slice(0, r, 2), slice(1, r, 2))
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        places = (slice(0, r // 2), slice(r // 2, r))
    # float64 itself: an angle of 10^9 radians errs by 2^-23
    rel = 2.0 ** -22 + 6 * U + 2.0 ** -52 * np.abs(angle).max(initial=0)
    err = rel * abs(scale) * (np.abs(a) + np.abs(b))
    for at, v in zip(places, (a * c - b * s, a * s + b * c)):
        y[..., at] = v
        tol[..., at] = err
    return y, tol + half_step(dtype) * np.abs(y)


# ---------------------------------------------------------------- norms
def _norm_back(v, ev, g, eg, kind, eps):
    """The normalised rows n, and the gradient of v from that of n, each with its error, where v errs
    by ev and g by eg.  A sum over d values is taken in runs of at most d / 8 (a thread's own
    columns) and ten halvings; the gradient is rho (g - mean(g) - n mean(g n))."""
    d = v.shape[-1]
    k = d / 8 + 14
    mean = lambda x: x.mean(-1, keepdims=True)  # noqa: E731
    if kind == "layer":
        ev = ev + (k + 2) * U * mean(np.abs(v)) + mean(ev) + U * np.abs(v)
        v = v - mean(v)
    q = mean(v * v)
    eq = (k + 2) * U * q + 2 * mean(np.abs(v) * ev) + mean(ev * ev)
    rho = 1 / np.sqrt(q + eps)
    rel = 0.5 * eq / (q + eps) + 6 * U  # of rho
    n = v * rho
    en = ev * rho + np.abs(n) * (rel + 2 * U)
    along = mean(g * n)
    ealong = (k + 8) * U * mean(np.abs(g * n)) + mean(np.abs(g) * en + eg * np.abs(n)) \
        + np.abs(along) * 2 * rel
    mg = mean(g) if kind == "layer" else 0.0
    emg = (k + 2) * U * mean(np.abs(g)) + mean(eg) if kind == "layer" else 0.0
    back = rho * (g - mg - n * along)
    err = rho * (eg + emg + en * np.abs(along) + np.abs(n) * ealong
                 + 6 * U * (np.abs(g) + np.abs(mg) + np.abs(n * along))) + np.abs(back) * (rel + U)
    return n, en, back, err


def _row_sum(terms, errs):
    """A parameter's gradient: the sum over rows (all axes but the last), in any grouping."""
    rows = int(np.prod(terms.shape[:-1]))
    total = terms.reshape(rows, -1).sum(0)
    mag = np.abs(terms).reshape(rows, -1).sum(0)
    # a chain of additions is at most rows long, and ends in a few dozen more
    return total, errs.reshape(rows, -1).sum(0) + (rows + 64) * U * mag + U * np.abs(total)


def gated_norm_back(dy, x, gate, weight, bias, norm, activation, gate_first, eps, dtype):
    """{"dx": [B,H,L,d], "dgate": [B,L,H*d], "dweight", "dbias"} with their bounds."""
    dy, x, gate, w, b = map(f64, (dy, x, gate, weight, bias))
    B, H, L, d = x.shape
    v = x.transpose(0, 2, 1, 3)
    dy = dy.reshape(B, L, H, d)
    shape = lambda t, one: np.full((1, d), one) if t is None else \
        t.reshape(1, d) if t.size == d else t.reshape(H, d)  # noqa: E731
    w, b = shape(w, 1.0), shape(b, 0.0)
    a, ea, slope, es = 1.0, 0.0, 0.0, 0.0
    if gate is not None:
        z = gate.reshape(B, L, H, d)
        a, ea, _ = act(activation, z)
        s = sigmoid(z)
        rel = 3 * U * np.abs(z) + SFU + 4 * U  # of the sigmoid (and of 1 less it, absolutely)
        err = s * rel + TINY
        if activation == "silu":
            slope = s + z * s * (1 - s)
            es = err * (1 + np.abs(z)) + 4 * U * (s + np.abs(z) * s)
        elif activation == "sigmoid":
            slope, es = s * (1 - s), 2 * err + 2 * U * s
        else:
            slope, es = 1.0, 0.0
    if gate_first and gate is not None:
        g, eg = dy * w, U * np.abs(dy * w)
        n, en, u, eu = _norm_back(v * a, np.abs(v) * ea + U * np.abs(v * a), g, eg, norm, eps)
        dx, ex = u * a, eu * np.abs(a) + np.abs(u) * ea + U * np.abs(u * a)
        dz = u * v * slope
        ez = eu * np.abs(v * slope) + np.abs(u * v) * es + 3 * U * np.abs(dz)
        dw, ew, db, eb = dy * n, np.abs(dy) * en, dy, 0 * dy
    else:
        g0 = dy * a
        e0 = np.abs(dy) * ea + U * np.abs(g0)
        n, en, dx, ex = _norm_back(v, 0 * v, g0 * w, e0 * np.abs(w) + U * np.abs(g0 * w), norm, eps)
        dz = dy * (n * w + b) * slope
        ez = np.abs(dy) * ((en * np.abs(w) + 2 * U * (np.abs(n * w) + np.abs(b))) * np.abs(slope)
                           + np.abs(n * w + b) * es) + 3 * U * np.abs(dz)
        dw, ew, db, eb = g0 * n, np.abs(g0) * en + e0 * np.abs(n), g0, e0
    out = {"dx": (dx.transpose(0, 2, 1, 3),
                  (ex + half_step(dtype) * np.abs(dx)).transpose(0, 2, 1, 3))}
    if gate is not None:
        dz, ez = dz + 0 * v, ez + 0 * v
        out["dgate"] = (dz.reshape(B, L, H * d),
                        (ez + half_step(dtype) * np.abs(dz)).reshape(B, L, H * d))
    for name, t, e, p in (("dweight", dw, ew, weight), ("dbias", db, eb, bias)):
        if p is not None:
            wide = p.numel() == H * d
            t, e = (y.reshape(-1, H * d) if wide else y.reshape(-1, d) for y in (t + 0 * v, e + 0 * v))
            out[name] = _row_sum(t, e)
    return out


def residual_norm_back(dy, r, weight, dr, x, post_weight, scale, alpha, norm, eps, dtype, res_dtype):
    """{"dx", "dresidual", "dweight", "dbias", "dpost_weight", "dscale"} with their bounds."""
    dy, r, w, dr, x, p, s = map(f64, (dy, r, weight, dr, x, post_weight, scale))
    alpha = float(np.float32(alpha))
    g = dy if w is None else dy * w
    n, en, e, ee = _norm_back(r, 0 * r, g, U * np.abs(g), norm, eps)
    if dr is not None:
        e = e + dr
        ee = ee + U * np.abs(e)
    out = {"dresidual": (e, ee + half_step(res_dtype) * np.abs(e)),
           "dweight": _row_sum(dy * n, np.abs(dy) * en), "dbias": _row_sum(dy, 0 * dy)}
    f = alpha * (1.0 if s is None else s) * (1.0 if p is None else p)
    g = e * f
    eg = (ee + 4 * U * np.abs(e)) * np.abs(f)
    if p is None:
        dx, ex = g, eg
        u, eu = x, None if x is None else 0 * x
    else:
        nx, enx, dx, ex = _norm_back(x, 0 * x, g, eg, norm, eps)
        u, eu = nx * p, enx * np.abs(p) + U * np.abs(nx * p)
        t = e * alpha * (1.0 if s is None else s)
        et = (ee + 3 * U * np.abs(e)) * abs(alpha) * (1.0 if s is None else np.abs(s))
        out["dpost_weight"] = _row_sum(t * nx, et * np.abs(nx) + np.abs(t) * enx)
    if s is not None:
        t = alpha * e
        out["dscale"] = _row_sum(t * u, (abs(alpha) * ee + 2 * U * np.abs(t)) * np.abs(u)
                                 + np.abs(t) * eu)
    out["dx"] = (dx, ex + half_step(dtype) * np.abs(dx))
    return out


# ---------------------------------------------------------------- attention
def log_decay(kind, decay, B, H, L):
    """[B,H,L] log decays and the derivative of each by what is given."""
    if kind == "none":
        return np.zeros((B, H, L)), np.zeros((B, H, L))
    a = f64(decay)
    if kind == "head":
        return np.broadcast_to(a[None, :, None], (B, H, L)), np.ones((B, H, L))
    if kind == "token":
        return a, np.ones((B, H, L))
    return -np.logaddexp(0, a), -sigmoid(a)


def _walk(q, k, v, dO, la, S0, dSf):
    """One sequence: dq, dk, dv, d log a, dS0, token by token."""
    L, dk = q.shape
    dv = v.shape[1]
    S = np.zeros((dk, dv)) if S0 is None else S0.copy()
    before = np.empty((L, dk, dv))
    dq = np.empty_like(q)
    a = np.exp(la)
    for t in range(L):
        before[t] = S
        S = a[t] * S + np.outer(k[t], v[t])
        dq[t] = S @ dO[t]
    G = np.zeros((dk, dv)) if dSf is None else dSf.copy()
    dk_, dv_, da = np.empty_like(k), np.empty_like(v), np.empty(L)
    for t in range(L - 1, -1, -1):
        G = G + np.outer(q[t], dO[t])
        dk_[t], dv_[t] = G @ v[t], G.T @ k[t]
        da[t] = a[t] * (G * before[t]).sum()
        G = a[t] * G
    return dq, dk_, dv_, da, G


def chunk_back(q, k, v, dO, phi, kind, decay, S0, dSf, dtype, want_f32=True):
    """{"dq", "dk", "dv", "ddecay", "dS0"} with their bounds.  ``want_f32``: whether the call asks
    for ddecay or dS0, whose products then keep 24 bits."""
    q, k, v, dO, S0, dSf = map(f64, (q, k, v, dO, S0, dSf))
    B, H, L, dk = q.shape
    dv = v.shape[-1]
    la, slope = log_decay(kind, decay, B, H, L)
    if phi == "elu1":
        fq, fk = (np.where(x > 0, x + 1, np.exp(np.minimum(x, 0))) for x in (q, k))
        q1, k1 = (np.where(x > 0, 1.0, np.exp(np.minimum(x, 0))) for x in (q, k))
    else:
        fq, fk, q1, k1 = q, k, np.ones_like(q), np.ones_like(k)
    shapes = {"dq": dk, "dk": dk, "dv": dv}
    val = {n: np.empty((B, H, L, w)) for n, w in shapes.items()}
    mag = {n: np.empty((B, H, L, w)) for n, w in shapes.items()}
    da, ma = np.empty((B, H, L)), np.empty((B, H, L))
    g0, mg0 = np.empty((B, H, dk, dv)), np.empty((B, H, dk, dv))
    for b in range(B):
        for h in range(H):
            at = (b, h)
            ends = [None if s is None else s[at] for s in (S0, dSf)]
            val["dq"][at], val["dk"][at], val["dv"][at], da[at], g0[at] = _walk(
                fq[at], fk[at], v[at], dO[at], la[at], *ends)
            mag["dq"][at], mag["dk"][at], mag["dv"][at], ma[at], mg0[at] = _walk(
                *(np.abs(x[at]) for x in (fq, fk, v, dO)), la[at],
                *(None if s is None else np.abs(s) for s in ends))
            # pairs of a block of 64 tokens are counted as differences of sums over the block; the
            # pairs around a chunk come from chunk to chunk as differences of such sums
            inside = (np.abs(fq[at]) * mag["dq"][at] + np.abs(fk[at]) * mag["dk"][at]).sum(-1)
            for t in range(0, L, 64):
                ma[at][t:t + 64] += inside[t:t + 64].sum() / 16
    chunks = -(-L // 32)
    f32 = (64 + 3 * chunks) * 2.0 ** -23 + 4 * 2.0 ** -21
    exact = dtype == "f32" or (want_f32 and phi == "elu1")
    rel = f32 if exact else 1.02 * (4 if phi == "elu1" else 2) * BF16 + f32
    out = {}
    for n, d1 in (("dq", q1), ("dk", k1), ("dv", 1.0)):
        x = val[n] * d1
        out[n] = (x, mag[n] * d1 * (rel + 2 * SFU) + half_step(dtype) * np.abs(x))
    x, tol = da * slope, ma * np.abs(slope) * (f32 + 8 * U)
    if kind == "head":
        out["ddecay"] = (x.sum((0, 2)), tol.sum((0, 2)) + U * np.abs(x).sum((0, 2)) * 64)
    elif kind != "none":
        out["ddecay"] = (x, tol + U * np.abs(x))
    out["dS0"] = (g0, mg0 * f32 + U * np.abs(g0))
    return out
