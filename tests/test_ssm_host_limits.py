"""The state space block's operators without a GPU, at the ends of what the C ABI and the binding
accept.  Calls that must pass a check end in a later one: they ask for more blocks than a grid has,
which is refused before any launch (status 3)."""
import os

import pytest
import torch

from causal_linear_attention_chunkwise_gb300 import _native, api, build
from tests.test_ssm_host import P, _conv, _gated, _resid, _scan

FAR = 1 << 60  # behind every range of these calls; never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_native.LIB_PATH):
        build.build()
    return _native.load()


# ---------------------------------------------------------------- overlaps
def _q(k):
    return P + k * 0x100000


@pytest.mark.parametrize("kw", [
    dict(y=P + 0x10000), dict(y=P + 0x103fe), dict(bias=P + 0x20000), dict(lengths=P + 0x203fc),
    dict(sf=P + 0x10000), dict(sf=P + 0x40000, bias=P + 0x40080),
    dict(sf=P + 0x40000, lengths=P + 0x40000),
])
def test_conv_refuses_outputs_over_parameters(lib, kw):
    assert _conv(lib, **kw) == 1
    assert b"overlaps" in lib.la_last_error()


@pytest.mark.parametrize("kw", [
    dict(hf=_q(5)), dict(hf=_q(5) + 4080), dict(hf=_q(7), bias=_q(7) + 4080),
    dict(hf=_q(7), skip=_q(7)), dict(hf=_q(7), lengths=_q(7) + 16), dict(y=_q(5) + 2),
    dict(bias=_q(6)), dict(skip=_q(6) + 16), dict(lengths=_q(6) + 1020),
    dict(h0=_q(1), hf=_q(1)),               # the state in place, and x in it too
    dict(L=0, hf=_q(5)),
])
def test_scan_refuses_outputs_over_parameters(lib, kw):
    assert _scan(lib, **kw) == 1
    assert b"overlaps" in lib.la_last_error()


def test_scan_refuses_a_workspace_over_its_tensors(lib):
    at = {k: v << 40 for v, k in enumerate(["x", "dt", "Bm", "Cm", "A", "y", "h0", "hf", "bias",
                                            "skip", "lengths", "z"], 1)}
    big = dict(at, L=65536, D=1024, xs=1024, ds=1024, ys=1024, zs=1024)
    need = lib.la_selective_scan_fwd_workspace_bytes(1, 65536, 1024, 16, 1)
    assert need > 0
    for k, p in at.items():
        assert _scan(lib, ws=p, wsb=need, **big) == 1, k
        assert b"workspace overlaps" in lib.la_last_error(), k
        assert _scan(lib, ws=p - need + 16, wsb=need, **big) == 1, k
        assert b"workspace overlaps" in lib.la_last_error(), k


@pytest.mark.parametrize("kw", [dict(weight=P + 0x20000), dict(bias=P + 0x20010),
                                dict(weight=P + 0x21ff0, wh=8), dict(weight=P + 0x1f810, wh=8)])
def test_gated_norm_refuses_its_output_over_parameters(lib, kw):
    assert _gated(lib, **kw) == 1
    assert b"overlaps" in lib.la_last_error()


@pytest.mark.parametrize("out", [0x20000, 0x30000])
@pytest.mark.parametrize("name", ["post", "scale", "weight", "bias"])
def test_residual_norm_refuses_outputs_over_parameters(lib, name, out):
    for at in (out, out + 0x3f0, out - 0xf0):  # 1024 bytes of output, 256 of parameters
        assert _resid(lib, **{name: P + at}) == 1
        assert b"overlaps" in lib.la_last_error()


# ---------------------------------------------------------------- slices of one tensor
def test_interleaved_slices_are_accepted(lib):
    """Outputs in their own columns of the tensor that the inputs are slices of; one element
    further they are refused."""
    D = 1 << 20
    conv = dict(B=2, L=1 << 30, D=D, xs=2 * D, ys=2 * D, weight=FAR)
    assert _conv(lib, y=P + 2 * D, **conv) == 3, lib.la_last_error()
    for y in (P + 2 * D - 2, P + 2 * D + 2):
        assert _conv(lib, y=y, **conv) == 1 and b"overlaps" in lib.la_last_error()
    w = 3 * 1024  # z, y and x in rows of three
    scan = dict(B=(1 << 31) - 1, L=9, D=1024, xs=w, ds=1024, zs=w, ys=w, z=P, x=P + 4096,
                dt=FAR, Bm=FAR + (1 << 56), Cm=FAR + (2 << 56), A=FAR + (3 << 56))
    assert _scan(lib, y=P + 2048, **scan) == 3, lib.la_last_error()
    for y in (P + 2046, P + 2050):
        assert _scan(lib, y=y, **scan) == 1 and b"overlaps" in lib.la_last_error()
    gated = dict(B=(1 << 31) - 1, H=1, L=16, d=512, xh=512, xt=1024, xb=16 * 1024, ys=1024,
                 gate=None)
    assert _gated(lib, y=P + 1024, **gated) == 3, lib.la_last_error()
    for y in (P + 1022, P + 1026):
        assert _gated(lib, y=y, **gated) == 1 and b"overlaps" in lib.la_last_error()


# ---------------------------------------------------------------- sizes
def test_binding_refuses_sizes_past_32_bits():
    """Without memory behind them ("meta"): cut to 32 bits, these would be small calls."""
    new = lambda *s: torch.empty(s, device="meta")  # noqa: E731
    big = (1 << 32) + 3
    for B, L, D in [(big, 1, 4), (1, big, 4), (1, 1, big)]:
        x = new(B, L, D)
        with pytest.raises(ValueError, match="2.31"):
            api.la_causal_conv_fwd(x, new(D, 4))
        with pytest.raises(ValueError, match="2.31"):
            api.la_selective_scan_fwd(x, x, new(D, 2), new(B, L, 2), new(B, L, 2))
        with pytest.raises(ValueError, match="2.31"):
            api.la_gated_norm_fwd(x[:, None])
    x = new(2, 3, 4)
    with pytest.raises(ValueError, match="2.31"):
        api.la_causal_conv_fwd(x, new(4, big))
    with pytest.raises(ValueError, match="2.31"):
        api.la_selective_scan_fwd(x, x, new(4, big), new(2, 3, big), new(2, 3, big))
    with pytest.raises(ValueError, match="2.31"):
        api.la_selective_scan_fwd(x, x, new(4, 2), new(2, 3, big, 2), new(2, 3, big, 2))
    with pytest.raises(ValueError, match="2.31"):
        api.la_gated_norm_fwd(new(1, big, 2, 4))
    with pytest.raises(ValueError, match="2.31"):
        api.la_residual_norm_fwd(new(1, big))
