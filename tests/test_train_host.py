"""The training pass's operators without a GPU: the 64-bit references against values worked by hand,
against autograd and against differences, and the refusals of the C ABI and of the Python binding
before any device work."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

from causal_linear_attention_chunkwise_gb300 import _native, api, build
from tests import ssm_reference as R
from tests import train_reference as T

P = 0x100000  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_native.LIB_PATH):
        build.build()
    return _native.load()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


# ---------------------------------------------------------------- references
def test_rotary_reference_by_hand():
    x = torch.tensor([[[[1.0, 2.0, 3.0, 4.0, 9.0]]]])
    f = torch.tensor([math.pi / 2, math.pi], dtype=torch.float32)
    one = torch.tensor([[1]])
    y, _ = T.rotary(x, f, one, 1.0, False, False, "f32")  # pairs (1,3) by 90, (2,4) by 180 degrees
    assert np.allclose(y[0, 0, 0], [-3, -2, 1, -4, 9], atol=1e-6)
    y, _ = T.rotary(x, f, one, 2.0, True, False, "f32")   # pairs (1,2) and (3,4), twice as long
    assert np.allclose(y[0, 0, 0], [-4, 2, -6, -8, 9], atol=1e-6)
    back, _ = T.rotary(torch.from_numpy(y), f, one, 0.5, True, True, "f32")
    assert np.allclose(back, x.numpy(), atol=1e-6)


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("gate_first", [False, True])
@pytest.mark.parametrize("activation", ["silu", "sigmoid", "none"])
@pytest.mark.parametrize("shared", [False, True])
def test_gated_norm_reference_is_autograd_of_the_forward(norm, gate_first, activation, shared):
    g = _gen(1)
    B, H, L, d = 2, 3, 4, 6
    x, gate = torch.randn(B, H, L, d, generator=g), torch.randn(B, L, H * d, generator=g)
    w, b = torch.rand(d if shared else H * d, generator=g), torch.randn(d if shared else H * d, generator=g)
    dy = torch.randn(B, L, H * d, generator=g)
    leaves = [t.double().requires_grad_(True) for t in (x, gate, w, b)]
    X, Z, W, Bi = leaves
    a = {"silu": torch.nn.functional.silu, "sigmoid": torch.sigmoid, "none": lambda t: t}[activation](Z)
    a = a.view(B, L, H, d)
    v = X.permute(0, 2, 1, 3)
    per = lambda t: t if shared else t.view(H, d)  # noqa: E731

    def normed(t):
        t = t - t.mean(-1, keepdim=True) if norm == "layer" else t
        return t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-5)

    y = normed(v * a) * per(W) + per(Bi) if gate_first else (normed(v) * per(W) + per(Bi)) * a
    want = torch.autograd.grad(y, leaves, dy.double().view(B, L, H, d))
    got = T.gated_norm_back(dy, x, gate, w, b, norm, activation, gate_first, 1e-5, "f32")
    for name, ref in zip(("dx", "dgate", "dweight", "dbias"), want):
        assert np.allclose(got[name][0], ref.numpy(), rtol=1e-9, atol=1e-11), name


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("scaled", [False, True])
def test_residual_norm_reference_is_autograd_of_the_forward(norm, post, scaled):
    g = _gen(2)
    x, res, dy, dr = (torch.randn(5, 7, generator=g).double() for _ in range(4))
    w, b, p, s = (torch.rand(7, generator=g).double() + 0.5 for _ in range(4))
    leaves = [t.clone().requires_grad_(True) for t in (x, res, w, b, p, s)]
    X, Rs, W, Bi, Pw, Sc = leaves

    def normed(t):
        t = t - t.mean(-1, keepdim=True) if norm == "layer" else t
        return t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-5)

    u = normed(X) * Pw if post else X
    r = Rs + 0.5 * (u * Sc if scaled else u)
    y = normed(r) * W + Bi
    want = dict(zip(("dx", "dresidual", "dweight", "dbias", "dpost_weight", "dscale"),
                    torch.autograd.grad((y, r), leaves, (dy, dr), allow_unused=True)))
    got = T.residual_norm_back(dy, r, w, dr, x, p if post else None, s if scaled else None, 0.5,
                               norm, 1e-5, "f32", "f32")
    for name, (val, _) in got.items():
        assert np.allclose(val, want[name].numpy(), rtol=1e-9, atol=1e-11), name
    assert ("dpost_weight" in got) == post and ("dscale" in got) == scaled


def _attention(kind, seed, L=7, dk=16, dv=32, states=True):
    g = _gen(seed)
    q, k = (0.3 * torch.randn(2, 2, L, dk, generator=g) for _ in range(2))
    v, dO = (torch.randn(2, 2, L, dv, generator=g) for _ in range(2))
    decay = {"none": None, "head": -torch.rand(2, generator=g),
             "token": -torch.rand(2, 2, L, generator=g),
             "logit": torch.randn(2, 2, L, generator=g)}[kind]
    S0, dSf = (torch.randn(2, 2, dk, dv, generator=g) if states else None for _ in range(2))
    return q, k, v, dO, decay, S0, dSf


@pytest.mark.parametrize("kind", ["none", "head", "token", "logit"])
@pytest.mark.parametrize("phi", ["identity", "elu1"])
def test_attention_reference_is_autograd_of_the_recurrence(kind, phi):
    q, k, v, dO, decay, S0, dSf = _attention(kind, 3)
    leaves = [t.double().requires_grad_(True) for t in (q, k, v, S0)]
    Q, K, V, S = leaves
    if decay is not None:
        leaves.append(decay.double().requires_grad_(True))
    f = (lambda x: torch.nn.functional.elu(x) + 1) if phi == "elu1" else (lambda x: x)
    O = []
    for t in range(q.shape[2]):
        a = {"none": lambda: 1.0, "head": lambda: torch.exp(leaves[-1])[None, :, None, None],
             "token": lambda: torch.exp(leaves[-1][:, :, t])[..., None, None],
             "logit": lambda: torch.sigmoid(-leaves[-1][:, :, t])[..., None, None]}[kind]()
        S = a * S + f(K)[:, :, t, :, None] * V[:, :, t, None, :]
        O.append((f(Q)[:, :, t, :, None] * S).sum(-2))
    want = torch.autograd.grad((torch.stack(O, 2), S), leaves, (dO.double(), dSf.double()))
    got = T.chunk_back(q, k, v, dO, phi, kind, decay, S0, dSf, "f32")
    for name, ref in zip(("dq", "dk", "dv", "dS0", "ddecay"), want):
        assert np.allclose(got[name][0], ref.numpy(), rtol=1e-9, atol=1e-11), name


def test_attention_reference_against_differences():
    """<dO, O> + <dSf, S> moves with each input as the gradients say."""
    import oracle
    q, k, v, dO, decay, S0, dSf = _attention("logit", 4, L=5)
    got = T.chunk_back(q, k, v, dO, "elu1", "logit", decay, S0, dSf, "f32")

    def loss(**kw):
        a = dict(q=q, k=k, v=v, decay=decay, S0=S0)
        a.update(kw)
        O, S = oracle.recurrent(a["q"], a["k"], a["v"], phi="elu1", decay_kind="logit",
                                decay=a["decay"], S0=a["S0"])
        return (np.asarray(O) * dO.double().numpy()).sum() + (np.asarray(S) * dSf.double().numpy()).sum()

    g = _gen(5)
    for name, key, t in (("q", "dq", q), ("k", "dk", k), ("v", "dv", v), ("decay", "ddecay", decay),
                         ("S0", "dS0", S0)):
        step = 2.0 ** -10 * torch.randn(t.shape, generator=g).sign()
        diff = loss(**{name: t + step}) - loss(**{name: t - step})
        moved = ((t + step).double() - (t - step).double()).numpy()
        # the third derivative's share: a step of 2^-10, cubed, against values of order 100
        assert abs(diff - (got[key][0] * moved).sum()) < 1e-4, name


@pytest.mark.parametrize("mistake", ["late", "slope", "decay", "mask", "state"])
def test_attention_bound_sees_mistakes(mistake):
    """The elementwise bound is far below what a wrong recurrence gives, in bf16 too."""
    q, k, v, dO, decay, S0, dSf = _attention("token", 6, L=20)
    ref = T.chunk_back(q, k, v, dO, "identity", "token", decay, S0, dSf, "bf16")
    bad = dict(q=q, k=k, v=v, dO=dO, phi="identity", kind="token", decay=decay, S0=S0, dSf=dSf,
               dtype="bf16")
    if mistake == "late":
        bad["dO"] = dO.roll(1, 2)
    elif mistake == "slope":
        bad["phi"] = "elu1"
    elif mistake == "decay":
        bad["decay"] = decay.roll(1, 2)
    elif mistake == "mask":
        bad["v"] = v.flip(2)
    else:
        bad["S0"] = None
        bad["dSf"] = None
    got = T.chunk_back(**bad)
    for name in ("dq", "dk"):
        with pytest.raises(AssertionError):
            R.check(torch.from_numpy(got[name][0]), ref[name], name)


# ---------------------------------------------------------------- frequencies
def test_frequencies_plain_linear_ntk():
    f, s = api.la_rotary_frequencies(8, 10000.0)
    assert s == 1.0 and torch.equal(f, (10000.0 ** (-torch.arange(4).double() / 4)).float())
    lin, _ = api.la_rotary_frequencies(8, 10000.0, "linear", 4.0)
    assert torch.equal(lin, (10000.0 ** (-torch.arange(4).double() / 4) / 4).float())
    ntk, _ = api.la_rotary_frequencies(8, 10000.0, "ntk", 4.0)
    assert ntk[0] == 1.0 and math.isclose(ntk[3], f[3] / 4, rel_tol=1e-6)  # the slowest: by factor
    one, _ = api.la_rotary_frequencies(2, 10000.0, "ntk", 4.0)
    assert one.tolist() == [1.0]


def test_frequencies_yarn():
    f, _ = api.la_rotary_frequencies(64, 10000.0)
    y, s = api.la_rotary_frequencies(64, 10000.0, "yarn", 8.0, trained_length=4096.0)
    turns = 4096 * f.double() / (2 * math.pi)
    assert math.isclose(s, 1 + 0.1 * math.log(8), rel_tol=1e-7)
    assert torch.equal(y[turns >= 32.01], f[turns >= 32.01])
    slow = turns <= 0.99
    assert slow.any() and torch.allclose(y[slow], f[slow] / 8, rtol=1e-6)
    between = (turns > 1.01) & (turns < 31.9)
    assert ((y[between] < f[between]) & (y[between] > f[between] / 8)).all()


@pytest.mark.parametrize("args", [
    dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=-2), dict(base=0.0), dict(base=math.inf),
    dict(scaling="linear", factor=0.5), dict(scaling="ntk", factor=math.nan),
    dict(scaling="yarn", factor=2.0), dict(scaling="yarn", factor=2.0, trained_length=10.0, fast=1.0),
])
def test_frequencies_refusals(args):
    with pytest.raises(api.LAError):
        api.la_rotary_frequencies(**{"rotary_dim": 8, **args})


# ---------------------------------------------------------------- C ABI refusals
def _rotary(lib, fn="la_rotary_fwd", **kw):
    a = dict(q=P, qb=8 * 64, qh=64, qt=128, Hq=2, k=None, kb=0, kh=0, kt=0, Hk=0, dtype=1, B=1, L=4,
             d=64, rot=64, inter=0, f=P + 0x10000, scale=1.0, pos=None, off=None, n=None,
             qo=P + 0x20000, qob=512, qoh=256, qot=64, ko=None, kob=0, koh=0, kot=0, stream=None)
    a.update(kw)
    return getattr(lib, fn)(*a.values())


@pytest.mark.parametrize("fn", ["la_rotary_fwd", "la_rotary_bwd"])
@pytest.mark.parametrize("kw,status", [
    (dict(dtype=5), 1), (dict(B=-1), 1), (dict(d=0), 1), (dict(rot=0), 1), (dict(rot=66), 1),
    (dict(rot=63), 1), (dict(d=16386), 2), (dict(Hq=20000), 2), (dict(L=2 ** 30 + 1), 2),
    (dict(q=None), 1), (dict(qo=None), 1), (dict(f=None), 1), (dict(q=P + 1), 1),
    (dict(f=P + 0x10002), 1), (dict(off=P + 0x30001), 1), (dict(pos=P + 0x30002), 1),
    (dict(n=P + 0x30003), 1), (dict(qt=-128), 1),
    (dict(qot=0), 1), (dict(qoh=64), 1),                    # two elements in one place
    (dict(qo=P, qob=512, qoh=256, qot=64), 1),               # in place with other strides
    (dict(qo=P + 64), 1), (dict(qo=P + 0x10000 - 64), 1),    # over the input, over the frequencies
    (dict(k=P + 0x40000, kb=512, kh=64, kt=128, Hk=2), 1),   # k without k_out
    (dict(k=P + 0x40000, kb=512, kh=64, kt=128, Hk=2, ko=P + 0x20100, kob=512, koh=256, kot=64), 1),
    (dict(k=P + 0x40000, kb=512, kh=64, kt=128, Hk=2, ko=P + 128, kob=512, koh=256, kot=64), 1),
    (dict(B=0, q=None), 0), (dict(L=0, q=None), 0), (dict(Hq=0, q=None), 0),
])
def test_rotary_refusals(lib, fn, kw, status):
    assert _rotary(lib, fn, **kw) == status, lib.la_last_error()


def _chunk(lib, **kw):
    a = dict(q=P, k=P + 0x100000, v=P + 0x200000, dtype=1, B=1, H=2, L=64, dk=64, dv=64, chunk=64,
             kind=0, decay=None, S0=None, dO=P + 0x300000, dSf=None, dq=P + 0x400000,
             dk_=P + 0x500000, dv_=P + 0x600000, dd=None, dS0=None, ws=P + 0x1000000, n=1 << 24,
             stream=None)
    a.update(kw)
    return lib.la_chunk_bwd(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), 1), (dict(B=-1), 1), (dict(L=-1), 1), (dict(dk=0), 1), (dict(chunk=0), 1),
    (dict(kind=4), 1), (dict(dk=48), 2), (dict(dv=256), 2), (dict(chunk=65), 2),
    (dict(L=2 ** 30 + 1), 2), (dict(B=2 ** 20, H=2 ** 12), 2),
    (dict(q=None), 1), (dict(dO=None), 1), (dict(dv_=None), 1), (dict(q=P + 8), 1),
    (dict(dk_=P + 0x500004), 1), (dict(S0=P + 0x700008), 1), (dict(dS0=P + 0x700004), 1),
    (dict(kind=1), 1), (dict(dd=P + 0x800000), 1),           # a decay kind without decays, and back
    (dict(kind=2, decay=P + 0x800002), 1), (dict(kind=2, decay=P + 0x800000, dd=P + 0x900001), 1),
    (dict(dq=P), 1), (dict(dk_=P + 0x100010), 1), (dict(dv_=P + 0x400000), 1),
    (dict(dS0=P + 0x700000, S0=P + 0x700000), 1), (dict(dS0=P + 0x700000, dSf=P + 0x700000), 1),
    (dict(kind=2, decay=P + 0x800000, dd=P + 0x800000), 1),
    (dict(ws=None), 1), (dict(n=16), 1), (dict(ws=P + 0x1000008), 1), (dict(ws=P + 0x300000), 1),
    (dict(ws=P + 0x400010), 1),
    (dict(B=0, q=None), 0), (dict(L=0, q=None), 0), (dict(H=0, q=None), 0),
])
def test_chunk_bwd_refusals(lib, kw, status):
    assert _chunk(lib, **kw) == status, lib.la_last_error()


def test_chunk_bwd_workspace_query(lib):
    ask = lib.la_chunk_bwd_workspace_bytes
    for bad in ((0, 1, 64, 64, 64, 64, 1), (1, 1, 64, 48, 64, 64, 1), (1, 1, 64, 64, 64, 65, 1),
                (1, 1, 64, 64, 64, 64, 3), (1, 1, 2 ** 30 + 1, 64, 64, 64, 1),
                (2 ** 20, 2 ** 12, 64, 64, 64, 64, 1)):
        assert ask(*bad) == 0
    # the shares of ddecay alone are three to five floats a token; states come in whole pairs
    for B, H, L, d, dt in ((1, 1, 1, 16, 0), (4, 16, 4096, 64, 1), (2, 32, 8192, 128, 1),
                           (1, 16, 32768, 128, 1), (3, 5, 777, 128, 0), (1, 1, 1 << 20, 64, 1)):
        need = ask(B, H, L, d, d, 64, dt)
        assert need >= 12 * B * H * L and need < 64 * B * H * (L + 128) + (1 << 34)


def _gated(lib, **kw):
    a = dict(dy=P, dys=128, x=P + 0x10000, xb=512, xh=256, xt=64, gate=P + 0x20000, gs=128, dtype=1,
             B=1, H=2, L=4, d=64, norm=0, act=1, first=0, w=P + 0x30000, b=None, wh=1, eps=1e-5,
             dx=P + 0x40000, dxb=512, dxh=256, dxt=64, dg=P + 0x50000, dgs=128, dw=P + 0x60000,
             db=None, ws=P + 0x100000, n=1 << 20, stream=None)
    a.update(kw)
    return lib.la_gated_norm_bwd(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), 1), (dict(L=-1), 1), (dict(d=0), 1), (dict(norm=2), 1), (dict(act=3), 1),
    (dict(eps=-1.0), 1), (dict(eps=math.nan), 1), (dict(d=16385, wh=1), 2), (dict(H=70000), 2),
    (dict(wh=3), 1), (dict(dys=127), 1), (dict(gs=100), 1), (dict(dgs=100), 1), (dict(xt=-1), 1),
    (dict(dxt=0), 1), (dict(dxh=32), 1), (dict(dy=None), 1), (dict(x=None), 1), (dict(dx=None), 1),
    (dict(dg=None), 1), (dict(gate=None), 1), (dict(x=P + 0x10001), 1), (dict(w=P + 0x30004), 1),
    (dict(dw=P + 0x60008), 1), (dict(dx=P), 1), (dict(dx=P + 0x20000), 1), (dict(dg=P + 0x10000), 1),
    (dict(dg=P + 2), 1), (dict(dx=P + 0x50000), 1), (dict(dw=P + 0x30000), 1), (dict(dw=P), 1),
    (dict(b=P + 0x70000, db=P + 0x60010), 1), (dict(dx=P + 0x10000, dxb=512, dxh=64, dxt=128), 1),
    (dict(ws=None), 1), (dict(n=8), 1), (dict(ws=P + 0x100004), 1), (dict(ws=P + 0x40000), 1),
    (dict(B=0, dw=None), 0),
])
def test_gated_norm_bwd_refusals(lib, kw, status):
    assert _gated(lib, **kw) == status, lib.la_last_error()


def _resid(lib, **kw):
    a = dict(dy=P, dtype=1, r=P + 0x10000, dr=P + 0x20000, res=1, x=P + 0x30000, rows=4, D=64,
             pw=P + 0x40000, sc=P + 0x41000, alpha=1.0, w=P + 0x42000, norm=0, eps=1e-5,
             dx=P + 0x50000, dres=P + 0x60000, dw=P + 0x70000, db=P + 0x71000, dp=P + 0x72000,
             ds=P + 0x73000, ws=P + 0x100000, n=1 << 20, stream=None)
    a.update(kw)
    return lib.la_residual_norm_bwd(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), 1), (dict(dtype=0, res=1), 1), (dict(res=7), 1), (dict(rows=-1), 1),
    (dict(D=0), 1), (dict(norm=2), 1), (dict(eps=-1.0), 1), (dict(D=16385), 2),
    (dict(dy=None), 1), (dict(r=None), 1), (dict(dx=None), 1), (dict(x=None), 1),
    (dict(pw=None), 1), (dict(sc=None), 1),                   # gradients of what is not there
    (dict(x=None, pw=None, dp=None), 1),                      # dscale needs x
    (dict(dy=P + 1), 1), (dict(r=P + 0x10001), 1), (dict(w=P + 0x42004), 1), (dict(dw=P + 0x70004), 1),
    (dict(dx=P + 2), 1), (dict(dx=P + 0x10000), 1), (dict(dx=P + 0x20000), 1), (dict(dres=P), 1),
    (dict(dres=P + 0x10000), 1), (dict(dres=P + 0x20002), 1), (dict(dres=P + 0x50000), 1),
    (dict(dw=P + 0x42000), 1), (dict(db=P + 0x70010), 1), (dict(ds=P + 0x30000), 1),
    (dict(ws=None), 1), (dict(n=8), 1), (dict(ws=P + 0x100008), 1), (dict(ws=P + 0x70000), 1),
    (dict(rows=0, dw=None, db=None, dp=None, ds=None), 0),
])
def test_residual_norm_bwd_refusals(lib, kw, status):
    assert _resid(lib, **kw) == status, lib.la_last_error()


# ---------------------------------------------------------------- binding refusals
def test_binding_refusals_before_the_library():
    t = torch.zeros
    f = t(32)
    with pytest.raises(ValueError):  # k of another head size
        api.la_rotary_fwd(t(1, 2, 4, 64), t(1, 2, 4, 32), f)
    with pytest.raises(ValueError):  # frequencies that are not fp32
        api.la_rotary_fwd(t(1, 2, 4, 64), None, f.double())
    with pytest.raises(ValueError):  # the last axis strided
        api.la_rotary_fwd(t(1, 2, 4, 128)[..., ::2], None, f)
    with pytest.raises(ValueError):
        api.la_rotary_fwd(t(1, 2, 4, 64), None, f, offsets=t(1))
    with pytest.raises(ValueError):
        api.la_rotary_fwd(t(1, 2, 4, 64), None, f, positions=t(1, 3, dtype=torch.int32))
    with pytest.raises(ValueError):  # on the host
        api.la_rotary_fwd(t(1, 2, 4, 64), None, f)
    q = t(1, 2, 4, 64)
    with pytest.raises(ValueError):  # a decay without its kind, and back
        api.la_chunk_bwd(q, q, q, q, decay=t(1, 2, 4))
    with pytest.raises(ValueError):
        api.la_chunk_bwd(q, q, q, q, decay_kind="token")
    with pytest.raises(ValueError):
        api.la_chunk_bwd(q, q, q, q, decay_kind="head", decay=t(1, 2, 4))
    with pytest.raises(ValueError):
        api.la_chunk_bwd(q, q, q.transpose(1, 2), q)
    with pytest.raises(ValueError):
        api.la_chunk_bwd(q, q, q, q.bfloat16())
    with pytest.raises(ValueError):
        api.la_chunk_bwd(q, q, q, q, S0=t(1, 2, 64, 32))
    x, dy = t(1, 2, 4, 8), t(1, 4, 16)
    with pytest.raises(ValueError):
        api.la_gated_norm_bwd(dy, x, None, t(9))
    with pytest.raises(ValueError):
        api.la_gated_norm_bwd(t(1, 4, 15), x)
    with pytest.raises(ValueError):
        api.la_gated_norm_bwd(dy, x, dgate=dy)
    with pytest.raises(ValueError):
        api.la_residual_norm_bwd(t(3, 8), t(3, 7))
    with pytest.raises(ValueError):
        api.la_residual_norm_bwd(t(3, 8), t(3, 8), weight=t(7))
    with pytest.raises(ValueError):
        api.la_residual_norm_bwd(t(3, 8), t(3, 8))
