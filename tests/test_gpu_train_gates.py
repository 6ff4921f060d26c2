"""The gated norm's backward pass with gates far from zero, where a sigmoid's slope s (1 - s) is a
small number on either side.  Needs a GB300."""
import numpy as np
import pytest
import torch

from causal_linear_attention_chunkwise_gb300 import api
from tests import train_reference as T
from tests.ssm_reference import SFU, U, check, f64

pytestmark = pytest.mark.gpu

NAN = float("nan")


def complement(z):
    """1 - sigmoid(z) without a difference."""
    return np.exp(-np.logaddexp(0, z))


@pytest.mark.parametrize("gate_first", [False, True])
@pytest.mark.parametrize("lo,hi", [(8, 20), (-20, -8), (20, 80), (-80, -20)])
@pytest.mark.parametrize("d", [64, 6, 1040])
def test_slope_of_far_sigmoid_gates(d, lo, hi, gate_first):
    """dgate in fp32 is its value up to rounding, however small the slope.  Relative errors: the
    exponent -z log2 e takes a rounding and log2 e's own, 2 U |z| in e^-z; the exponential and the
    reciprocal SFU each; the sum, the product and that of s and 1 - s U each, with s and 1 - s
    both off by what e^-z is."""
    B, H, L = 2, 3, 17
    g = torch.Generator().manual_seed(d + lo)
    x, dy = torch.randn(B, H, L, d, generator=g), torch.randn(B, L, H * d, generator=g)
    gate = lo + (hi - lo) * torch.rand(B, L, H * d, generator=g)
    w = torch.rand(d, generator=g) + 0.5
    got = api.la_gated_norm_bwd(dy.cuda(), x.cuda(), gate.cuda(), w.cuda(), activation="sigmoid",
                                gate_first=gate_first)[1]
    z, X, Y = (f64(t).reshape(B, L, H, d) for t in (gate, x.permute(0, 2, 1, 3), dy))
    W = f64(w)
    s, rest = complement(-z), complement(z)
    slope = s * rest
    rel = 2 * (2 * U * np.abs(z) + 2 * SFU + 2 * U) + 2 * U
    if gate_first:
        ea = s * rel / 2
        _, _, u, eu = T._norm_back(X * s, np.abs(X) * ea + U * np.abs(X * s), Y * W,
                                   U * np.abs(Y * W), "rms", 1e-5)
        dz = u * X * slope
        tol = eu * np.abs(X) * slope + np.abs(dz) * (rel + 3 * U)
    else:
        n, en, _, _ = T._norm_back(X, 0 * X, Y, 0 * Y, "rms", 1e-5)
        dz = Y * n * W * slope
        tol = np.abs(Y) * en * W * slope + np.abs(dz) * (rel + 5 * U)
    check(got, (dz.reshape(B, L, H * d), tol.reshape(B, L, H * d) + 2.0 ** -126), "dgate")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("activation", ["sigmoid", "silu"])
@pytest.mark.parametrize("d", [64, 7])
def test_gates_at_the_ends(d, activation, dtype):
    """Gates whose exponential overflows or vanishes have slopes of 0 or 1; a NaN gate
    spoils its own row alone."""
    z = torch.tensor([-1e30, -500.0, -200.0, -129.0, 129.0, 200.0, 500.0, 1e30], device="cuda")
    L = z.numel()
    x = torch.ones(1, 1, L, d, device="cuda", dtype=dtype)
    dy = torch.ones(1, L, d, device="cuda", dtype=dtype)
    gate = z[None, :, None].expand(1, L, d).to(dtype).contiguous()
    dx, dz, _, _ = api.la_gated_norm_bwd(dy, x, gate, activation=activation, eps=0.0)
    want = 0.0 if activation == "sigmoid" else 1.0
    assert (dz[0, :4] == 0).all()
    # the norm of a row of ones: the mean's factor, the sum, the root and two products
    assert ((dz[0, 4:].float() - want).abs() <= want * 2.0 ** -20).all()
    assert torch.isfinite(dx[0, 0, :4]).all()
    gate[0, 2] = NAN
    dx2, dz2, _, _ = api.la_gated_norm_bwd(dy, x, gate, activation=activation, eps=0.0)
    assert torch.isnan(dz2[0, 2]).all() and torch.isnan(dx2[0, 0, 2]).all()
    keep = [i for i in range(L) if i != 2]
    assert torch.equal(dz2[0, keep], dz[0, keep]) and torch.equal(dx2[0, 0, keep], dx[0, 0, keep])
