"""Tokens that nearly reset the state: their decay's gradient is a sum of the pairs that they lie
between, so much smaller than their neighbours' that a difference of those would leave little of
it.  Needs a GB300."""
import numpy as np
import pytest
import torch

from causal_linear_attention_chunkwise_gb300 import api
from tests import train_reference as T
from tests.ssm_reference import U, check

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
INF = float("inf")


@pytest.fixture(autouse=True)
def _identity():
    api.la_set_feature_map("identity")
    yield
    api.la_set_feature_map("identity")


def reference(q, k, v, dO, phi, la, S0, dSf):
    """d log a of every token, and the sum of the magnitudes of the pairs that it lies between."""
    q, k, v, dO, S0, dSf = (None if t is None else T.f64(t) for t in (q, k, v, dO, S0, dSf))
    if phi == "elu1":
        q, k = (np.where(x > 0, x + 1, np.exp(np.minimum(x, 0))) for x in (q, k))
    da, mag = np.empty(la.shape), np.empty(la.shape)
    for at in np.ndindex(*la.shape[:2]):
        ends = [None if s is None else s[at] for s in (S0, dSf)]
        da[at] = T._walk(q[at], k[at], v[at], dO[at], la[at], *ends)[3]
        mag[at] = T._walk(*(np.abs(x[at]) for x in (q, k, v, dO)), la[at],
                          *(None if s is None else np.abs(s) for s in ends))[3]
    return da, mag


def run(B, H, L, dk, dv, dtype, phi, kind, resets, states, seed=0):
    """``resets``: {token: its log decay}; all others decay by e^-0.05."""
    g = torch.Generator().manual_seed(seed)
    q, k = (0.3 * torch.randn(B, H, L, dk, generator=g) for _ in range(2))
    v, dO = (torch.randn(B, H, L, dv, generator=g) for _ in range(2))
    q, k, v, dO = (t.to(DT[dtype]) for t in (q, k, v, dO))
    S0, dSf = (torch.randn(B, H, dk, dv, generator=g) if states else None for _ in range(2))
    la = torch.full((B, H, L), -0.05) * (0.5 + torch.rand(B, H, L, generator=g))
    for t, a in resets.items():
        la[..., t] = a
    if kind == "logit":  # -softplus(x) = log a: x = log(1 / a - 1)
        decay = torch.where(la == -INF, INF, torch.log(torch.expm1(-la.double()))).float()
    else:
        decay = la
    la, slope = T.log_decay(kind, decay, B, H, L)
    api.la_set_feature_map(phi)
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    got = api.la_chunk_bwd(*map(cuda, (q, k, v, dO)), decay_kind=kind, decay=cuda(decay),
                           S0=cuda(S0), dS_final=cuda(dSf))[3]
    api.la_device_status()
    da, mag = reference(q, k, v, dO, phi, la, S0, dSf)
    # the counts of train_reference: products of 24 bits, over the pairs' own magnitudes alone
    f32 = (64 + 3 * -(-L // 32)) * 2.0 ** -23 + 4 * 2.0 ** -21
    val, tol = da * slope, mag * np.abs(slope) * (f32 + 9 * U)
    live = np.zeros(la.shape, bool)  # tokens of a reset's block of 32
    for t in resets:
        live[..., t // 32 * 32:t // 32 * 32 + 32] = True
    check(got, (val, tol), "ddecay", live)


@pytest.mark.parametrize("kind", ["token", "logit"])
@pytest.mark.parametrize("dtype,phi,dk,dv", [
    ("bf16", "identity", 64, 64), ("bf16", "identity", 128, 128), ("bf16", "identity", 16, 32),
    ("bf16", "elu1", 64, 64), ("bf16", "elu1", 64, 128), ("f32", "identity", 64, 64),
    ("f32", "identity", 128, 64), ("f32", "elu1", 128, 128), ("f32", "elu1", 32, 16)])
@pytest.mark.parametrize("states", [False, True])
def test_one_reset_in_several_chunks(dtype, phi, dk, dv, kind, states):
    """In the middle of a block, at its ends, at a chunk's, one after another, of several strengths."""
    run(1, 2, 700, dk, dv, dtype, phi, kind,
        {17: -10.0, 128: -10.0, 255: -8.0, 300: -4.0, 330: -12.0, 331: -6.0, 448: -30.0, 480: -10.0,
         600: -INF}, states)


@pytest.mark.parametrize("dtype,phi,dk,dv,L", [
    ("bf16", "identity", 64, 64, 64), ("bf16", "identity", 64, 64, 50), ("bf16", "elu1", 64, 64, 64),
    ("f32", "identity", 64, 64, 64), ("bf16", "identity", 128, 128, 64)])
def test_many_short_sequences(dtype, phi, dk, dv, L):
    run(5, 32, L, dk, dv, dtype, phi, "token", {5: -10.0, 33: -9.0, 40: -INF}, L == 50)


@pytest.mark.parametrize("dtype,phi", [("bf16", "identity"), ("f32", "identity"), ("bf16", "elu1")])
def test_resets_in_segments(dtype, phi):
    """One long sequence, which is cut; a reset every 97 tokens, as between packed documents."""
    run(1, 1, 3000, 64, 64, dtype, phi, "token", {t: -10.0 for t in range(50, 3000, 97)}, True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_reset_at_every_token(dtype):
    run(1, 2, 300, 64, 64, dtype, "identity", "token", {t: -9.0 for t in range(300)}, True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_reset_at_all_is_as_before(dtype):
    """Slow decays alone, and one just below what counts as strong: the bound of the pairs around a
    chunk as differences, which train_reference counts."""
    g = torch.Generator().manual_seed(3)
    B, H, L, d = 1, 2, 600, 64
    q, k, v, dO = (torch.randn(B, H, L, d, generator=g).mul_(0.4).to(DT[dtype]) for _ in range(4))
    la = -0.01 * torch.rand(B, H, L, generator=g)
    la[..., 200] = -3.4
    ref = T.chunk_back(q, k, v, dO, "identity", "token", la, None, None, dtype)
    got = api.la_chunk_bwd(q.cuda(), k.cuda(), v.cuda(), dO.cuda(), decay_kind="token",
                           decay=la.cuda())[3]
    check(got, ref["ddecay"], "ddecay")
