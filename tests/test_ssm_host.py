"""The state space block's operators without a GPU: the 64-bit references
against values worked by hand and against each other, and the refusals of the C
ABI and of the Python binding before any device work."""
import ctypes
import os

import numpy as np
import pytest
import torch

from causal_linear_attention_chunkwise_gb300 import _native, api, build
from tests import ssm_reference as R

P = 0x100000  # never dereferenced: validation fails first
LL = ctypes.c_longlong


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_native.LIB_PATH):
        build.build()
    return _native.load()


# ---------------------------------------------------------------- references
def test_conv_reference_by_hand():
    # one channel, W = 3, weights (1, 10, 100) over (x[t-2], x[t-1], x[t]), bias 0.5
    x = torch.tensor([[[1.0], [2.0], [3.0]]])
    st = torch.tensor([[[7.0], [8.0]]])
    (y, _), last = R.causal_conv(x, torch.tensor([[1.0, 10.0, 100.0]]), torch.tensor([0.5]),
                                 "none", st, None, "f32")
    assert y[0, :, 0].tolist() == [7 + 80 + 100 + 0.5, 8 + 10 + 200 + 0.5, 1 + 20 + 300 + 0.5]
    assert last[0, :, 0].tolist() == [2.0, 3.0]
    _, last = R.causal_conv(x, torch.tensor([[1.0, 10.0, 100.0]]), None, "none", st,
                            torch.tensor([1], dtype=torch.int32), "f32")
    assert last[0, :, 0].tolist() == [8.0, 1.0]


def test_scan_reference_by_hand():
    # one channel, one state, A = -1, delta = 0.5 then 0.25, no softplus
    one = lambda *v: torch.tensor(v).reshape(1, -1, 1)  # noqa: E731
    (y, _), (h, _) = R.selective_scan(
        one(2.0, 4.0), one(0.5, 0.25), torch.tensor([[-1.0]]), one(3.0, 1.0), one(1.0, -2.0),
        torch.tensor([10.0]), None, None, False, torch.tensor([[[8.0]]]), None, "f32")
    h1 = np.exp(-0.5) * 8 + 0.5 * 2 * 3
    h2 = np.exp(-0.25) * h1 + 0.25 * 4 * 1
    assert np.allclose(y[0, :, 0], [h1 + 20, -2 * h2 + 40], rtol=1e-14)
    assert np.allclose(h[0, 0, 0], h2, rtol=1e-14)


def test_scan_reference_is_linear_attention_when_the_decay_is_shared():
    """With A = -1 everywhere and no skip or gate the scan is the gated linear
    attention recurrence with alpha = exp(-delta) and values delta x."""
    import oracle
    g = torch.Generator().manual_seed(0)
    B, L, ch, N = 2, 9, 3, 16
    x, Bm, Cm = (torch.randn(B, L, k, generator=g) for k in (ch, N, N))
    # values delta x in 64 bits: the oracle takes fp32 inputs, so choose delta a power of two
    dt = torch.full((B, L, ch), 0.25)
    (y, _), (h, _) = R.selective_scan(x, dt, -torch.ones(ch, N), Bm, Cm, None, None, None, False,
                                      None, None, "f32")
    O, S = oracle.recurrent(Cm[:, None], Bm[:, None], (0.25 * x)[:, None], phi="identity",
                            decay_kind="token", decay=-dt[..., 0][:, None].contiguous())
    assert np.allclose(y, np.asarray(O)[:, 0], rtol=1e-12, atol=1e-12)
    assert np.allclose(h, np.asarray(S)[:, 0].transpose(0, 2, 1), rtol=1e-12, atol=1e-12)


def test_norm_references_against_torch():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(2, 3, 4, 10, generator=g).double()
    w, b = torch.rand(10, generator=g).double(), torch.randn(10, generator=g).double()
    gate = torch.randn(2, 4, 30, generator=g).double()
    y, _ = R.gated_norm(x, gate, w, b, "layer", "silu", False, 1e-5, "f32")
    ref = torch.nn.functional.layer_norm(x, (10,), w, b, 1e-5).permute(0, 2, 1, 3).reshape(2, 4, 30)
    assert np.allclose(y, ref * torch.nn.functional.silu(gate), rtol=1e-12)
    y, _ = R.gated_norm(x, gate, w, None, "rms", "sigmoid", True, 1e-5, "f32")
    v = x.permute(0, 2, 1, 3) * torch.sigmoid(gate).view(2, 4, 3, 10)
    ref = v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-5) * w
    assert np.allclose(y, ref.reshape(2, 4, 30), rtol=1e-12)
    (y, _), (r, _) = R.residual_norm(x, 2 * x, None, w, 0.5, None, None, "rms", 0.0, "f32", "f32")
    ref = 2 * x + 0.5 * w * x
    assert np.allclose(r, ref, rtol=1e-12)
    assert np.allclose(y, ref / torch.sqrt((ref * ref).mean(-1, keepdim=True)), rtol=1e-12)


@pytest.mark.parametrize("mistake", ["late", "softplus", "group", "gate", "skip"])
def test_scan_bound_sees_mistakes(mistake):
    """The elementwise bound is far below what a wrong recurrence gives."""
    g = torch.Generator().manual_seed(2)
    B, L, ch, N = 1, 12, 4, 5
    x, dt, z = (torch.randn(B, L, ch, generator=g) for _ in range(3))
    Bm, Cm = (torch.randn(B, L, 2, N, generator=g) for _ in range(2))
    A = -torch.rand(ch, N, generator=g) - 0.1
    D = torch.randn(ch, generator=g)
    args = dict(x=x, dt=dt, A=A, Bm=Bm, Cm=Cm, D=D, z=z, dt_bias=None, softplus=True, h0=None,
                lengths=None, dtype="f32")
    ref, _ = R.selective_scan(**args)
    bad = dict(args)
    if mistake == "late":
        bad["Cm"] = Cm.roll(1, 1)
    elif mistake == "softplus":
        bad["dt"] = dt + 1e-4
    elif mistake == "group":
        bad["Bm"] = Bm.flip(2)
    elif mistake == "gate":
        bad["z"] = None
    else:
        bad["D"] = D * (1 + 1e-4)
    (y, _), _ = R.selective_scan(**bad)
    with pytest.raises(AssertionError):
        R.check(torch.from_numpy(y), ref, "y")


# ---------------------------------------------------------------- C ABI refusals
def _conv(lib, **kw):
    a = dict(x=P, xs=64, dtype=1, B=1, L=8, D=64, W=4, weight=P + 0x10000, bias=None, act=1,
             lengths=None, state0=None, y=P + 0x20000, ys=64, sf=None, stream=None)
    a.update(kw)
    return lib.la_causal_conv_fwd(*a.values())


@pytest.mark.parametrize("kw,status,word", [
    (dict(dtype=7), 1, b"dtype"), (dict(B=-1), 1, b"sizes"), (dict(L=-3), 1, b"sizes"),
    (dict(L=(1 << 30) + 1), 2, b"2^30"),
    (dict(W=1), 2, b"width"), (dict(W=9), 2, b"width"), (dict(act=2), 1, b"activation"),
    (dict(xs=63), 1, b"stride"), (dict(ys=10), 1, b"stride"), (dict(weight=None), 1, b"non-null"),
    (dict(x=None), 1, b"non-null"), (dict(y=None), 1, b"non-null"), (dict(x=P + 1), 1, b"aligned"),
    (dict(weight=P + 0x10004), 1, b"16-byte"), (dict(y=P), 1, b"overlaps"),
    (dict(y=P + 256), 1, b"overlaps"), (dict(sf=P), 1, b"overlaps"),
    (dict(state0=P + 0x40000, sf=P + 0x40080), 1, b"overlaps"),
    (dict(sf=P + 0x20000), 1, b"overlaps"), (dict(lengths=P + 0x50002), 1, b"aligned"),
])
def test_conv_refusals(lib, kw, status, word):
    assert _conv(lib, **kw) == status
    assert word in lib.la_last_error()


def test_conv_slices_of_one_tensor_do_not_overlap(lib):
    """y may interleave with x in one wider tensor; only B = 0 keeps the call from launching."""
    assert _conv(lib, xs=128, ys=128, y=P + 128, B=0) == 0
    assert _conv(lib, xs=128, ys=128, y=P + 126) == 1
    assert b"overlaps" in lib.la_last_error()


def _scan(lib, **kw):
    q = lambda k: P + k * 0x100000  # noqa: E731
    a = dict(x=q(1), xs=64, dt=q(2), ds=64, z=None, zs=0, Bm=q(3), bs=16, Cm=q(4), cs=16, dtype=1,
             B=1, L=8, D=64, N=16, G=1, A=q(5), bias=None, sp=1, skip=None, h0=None, lengths=None,
             y=q(6), ys=64, hf=None, ws=None, wsb=0, stream=None)
    a.update(kw)
    return lib.la_selective_scan_fwd(*a.values())


@pytest.mark.parametrize("kw,status,word", [
    (dict(dtype=2), 1, b"dtype"), (dict(N=0), 1, b"sizes"), (dict(N=257, bs=257, cs=257), 2, b"N="),
    (dict(G=3, bs=48, cs=48), 2, b"groups"), (dict(G=0), 1, b"sizes"), (dict(D=-1), 1, b"sizes"),
    (dict(L=(1 << 30) + 1), 2, b"2^30"),
    (dict(xs=8), 1, b"stride"), (dict(bs=15), 1, b"stride"), (dict(G=2, bs=16, cs=32), 1, b"stride"),
    (dict(z=P, zs=63), 1, b"stride"), (dict(A=None), 1, b"non-null"), (dict(dt=None), 1, b"non-null"),
    (dict(A=P + 4), 1, b"16-byte"), (dict(h0=P + 8), 1, b"16-byte"), (dict(x=P + 1), 1, b"aligned"),
    (dict(y=P + 0x100000), 1, b"overlaps"), (dict(y=P + 0x300010), 1, b"overlaps"),
    (dict(h0=P, hf=P + 16), 1, b"overlaps"), (dict(hf=P + 0x500000), 0, None),
    (dict(hf=P + 0x200000), 1, b"overlaps"), (dict(hf=P + 0x600000), 1, b"overlaps"),
    (dict(lengths=P + 1), 1, b"lengths"),
])
def test_scan_refusals(lib, kw, status, word):
    if word is None:  # parameters are not compared with states: B = 0 ends the call first
        assert _scan(lib, B=0, **kw) == 0
        return
    assert _scan(lib, **kw) == status
    assert word in lib.la_last_error()


def test_scan_refuses_a_small_or_misaligned_workspace(lib):
    need = lib.la_selective_scan_fwd_workspace_bytes(1, 65536, 1024, 16, 1)
    big = dict(L=65536, D=1024, xs=1024, ds=1024, ys=1024, x=1 << 40, dt=2 << 40, Bm=3 << 40,
               Cm=4 << 40, y=6 << 40)
    if need:
        assert _scan(lib, ws=P, wsb=need - 1, **big) == 1 and b"workspace" in lib.la_last_error()
    assert _scan(lib, ws=P + 8, wsb=need, **big) == 1 and b"16-byte" in lib.la_last_error()
    for args in [(0, 9, 9, 16, 1), (1, 0, 9, 16, 1), (1, 9, 9, 300, 1), (1, 9, 9, 16, 2)]:
        assert lib.la_selective_scan_fwd_workspace_bytes(*args) == 0


def _gated(lib, **kw):
    a = dict(x=P, xb=4096, xh=512, xt=64, gate=P + 0x10000, gs=512, dtype=1, B=1, H=8, L=8, d=64,
             norm=0, act=1, first=0, weight=None, bias=None, wh=1, eps=1e-5, y=P + 0x20000, ys=512,
             stream=None)
    a.update(kw)
    return lib.la_gated_norm_fwd(*a.values())


@pytest.mark.parametrize("kw,status,word", [
    (dict(dtype=2), 1, b"dtype"), (dict(d=0), 1, b"sizes"), (dict(d=16385, ys=1 << 20, gs=1 << 20), 2, b"d="),
    (dict(norm=2), 1, b"norm"), (dict(act=3), 1, b"activation"), (dict(eps=-1.0), 1, b"eps"),
    (dict(eps=float("nan")), 1, b"eps"), (dict(wh=3), 1, b"weight_heads"), (dict(xt=-1), 1, b"stride"),
    (dict(ys=511), 1, b"stride"), (dict(gs=511), 1, b"stride"), (dict(x=None), 1, b"non-null"),
    (dict(y=None), 1, b"non-null"), (dict(gate=P + 0x10001), 1, b"aligned"),
    (dict(weight=P + 4), 1, b"16-byte"), (dict(y=P + 64), 1, b"overlaps"),
    (dict(y=P + 0x10000, ys=520), 1, b"overlaps"), (dict(y=P + 0x10002), 1, b"overlaps"),
    # one head, token major, rows 1024 apart: the other half of the rows is free, its own is not
    (dict(H=1, d=512, xh=7, xt=1024, xb=8192, ys=1024, y=P + 1022), 1, b"overlaps"),
    (dict(H=1, d=512, xh=7, xt=1024, xb=8192, ys=1024, y=P + 1024, eps=-1.0), 1, b"eps"),
])
def test_gated_norm_refusals(lib, kw, status, word):
    assert _gated(lib, **kw) == status
    assert word in lib.la_last_error()


def _resid(lib, **kw):
    a = dict(x=P, dtype=1, res=P + 0x10000, rd=1, rows=8, D=64, post=None, scale=None, alpha=1.0,
             weight=None, bias=None, norm=0, eps=1e-5, y=P + 0x20000, ro=P + 0x30000, stream=None)
    a.update(kw)
    return lib.la_residual_norm_fwd(*a.values())


@pytest.mark.parametrize("kw,status,word", [
    (dict(dtype=2), 1, b"dtype"), (dict(dtype=0, rd=1), 1, b"residual"), (dict(rd=5), 1, b"residual"),
    (dict(rows=-1), 1, b"sizes"), (dict(D=0), 1, b"sizes"), (dict(D=16385), 2, b"D="),
    (dict(norm=-1), 1, b"norm"), (dict(eps=float("nan")), 1, b"eps"), (dict(x=None), 1, b"non-null"),
    (dict(y=None), 1, b"non-null"), (dict(res=P + 0x10002, rd=0), 1, b"aligned"),
    (dict(scale=P + 2), 1, b"16-byte"), (dict(y=P + 2), 1, b"overlaps"),
    (dict(y=P + 0x10000), 1, b"overlaps"), (dict(ro=P), 1, b"overlaps"),
    (dict(ro=P + 0x20000), 1, b"overlaps"), (dict(ro=P + 0x10002), 1, b"overlaps"),
])
def test_residual_norm_refusals(lib, kw, status, word):
    assert _resid(lib, **kw) == status
    assert word in lib.la_last_error()


def test_empty_calls_are_no_ops(lib):
    assert _conv(lib, B=0, x=None, y=None) == 0
    assert _conv(lib, D=0, x=None, y=None) == 0
    assert _scan(lib, B=0, x=None, y=None) == 0
    assert _scan(lib, L=0, x=None, dt=None, Bm=None, Cm=None, y=None) == 0  # no final state asked
    assert _gated(lib, L=0, x=None, y=None) == 0
    assert _gated(lib, H=0, wh=0, x=None, y=None) == 0
    assert _resid(lib, rows=0, x=None, y=None) == 0


# ---------------------------------------------------------------- Python refusals
def test_binding_refuses_before_the_library():
    x = torch.zeros(2, 5, 8)
    w = torch.zeros(8, 4)
    with pytest.raises(ValueError, match="CUDA"):
        api.la_causal_conv_fwd(x, w)
    with pytest.raises(ValueError, match="weight"):
        api.la_causal_conv_fwd(x, torch.zeros(7, 4))
    with pytest.raises(ValueError, match="weight"):
        api.la_causal_conv_fwd(x, w.double())
    with pytest.raises(ValueError, match="lengths"):
        api.la_causal_conv_fwd(x, w, lengths=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="states"):
        api.la_causal_conv_fwd(x, w, state0=torch.zeros(2, 4, 8))
    with pytest.raises(ValueError, match="evenly"):
        api.la_causal_conv_fwd(torch.zeros(2, 9, 8)[:, :5], w)
    with pytest.raises(ValueError, match="contiguous"):
        api.la_causal_conv_fwd(torch.zeros(2, 5, 16)[..., ::2], w)
    A, bc = torch.zeros(8, 4), torch.zeros(2, 5, 4)
    with pytest.raises(ValueError, match="CUDA"):
        api.la_selective_scan_fwd(x, x, A, bc, bc)
    with pytest.raises(ValueError, match="dt"):
        api.la_selective_scan_fwd(x, x[:, :4], A, bc, bc)
    with pytest.raises(ValueError, match="Cm"):
        api.la_selective_scan_fwd(x, x, A, bc, bc[..., :3])
    with pytest.raises(ValueError, match="z must"):
        api.la_selective_scan_fwd(x, x, A, bc, bc, z=x.bfloat16())
    with pytest.raises(ValueError, match="h0"):
        api.la_selective_scan_fwd(x, x, A, bc, bc, h0=torch.zeros(2, 4, 8))
    o = torch.zeros(2, 3, 5, 8)
    with pytest.raises(ValueError, match="CUDA"):
        api.la_gated_norm_fwd(o)
    with pytest.raises(ValueError, match="gate"):
        api.la_gated_norm_fwd(o, gate=torch.zeros(2, 5, 8))
    with pytest.raises(ValueError, match="weight"):
        api.la_gated_norm_fwd(o, weight=torch.zeros(16))
    with pytest.raises(ValueError, match="one shape"):
        api.la_gated_norm_fwd(o, weight=torch.zeros(8), bias=torch.zeros(24))
    with pytest.raises(ValueError, match="last axis"):
        api.la_gated_norm_fwd(o.transpose(2, 3))
    with pytest.raises(ValueError, match="CUDA"):
        api.la_residual_norm_fwd(x)
    with pytest.raises(ValueError, match="one shape"):
        api.la_residual_norm_fwd(x, residual=x[:, :4])
    with pytest.raises(ValueError, match="weight"):
        api.la_residual_norm_fwd(x, weight=torch.zeros(5))
